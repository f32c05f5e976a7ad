"""Values at the edge in the attention layers' cache: infinities and NaN beside places that are
only copied, scales and scores far from one, and codes on a rounding tie.

Tolerances are derived where each test states them; u is the unit roundoff as in
test_attn_gpu.py (2^-24 fp32, 2^-8 bf16, 2^-11 fp16, 2^-22 for sums of tensor cores).
"""
import math

import numpy as np
import pytest
import torch

from test_attn_gpu import BF, F8, F32, attn, attn_problem, check_attn, new_pools, np64, rot_tables  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- places that are not rotated ------------------------------------------------


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.int32)


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("D,R", [(64, 0), (64, 16), (64, 48), (128, 0), (128, 32), (128, 96)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [9, 2500])
def test_append_copies_unrotated_places(attn, T, dt, D, R, interleaved):
    """Without a norm the places from R on are a copy, bit for bit: an infinity, a NaN or a
    negative zero among them stays where it is, in queries, keys and values."""
    Hq, Hkv = 4, 2
    g = torch.Generator().manual_seed(D + R)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dt)
    plain = x.clone()
    for t, value in ((0, float("inf")), (1, float("-inf")), (2, float("nan")), (3, -0.0)):
        for place in (R, R + 7, D - 1, D - 16):
            x[t, :, max(place, R)] = value
    x[4, :, R:] = -0.0
    x[5, :, R::2] = -0.0
    cos = sin = pos = None
    if R:
        cos, sin = (y.cuda() for y in rot_tables(3 * T, R))
        pos = torch.arange(T, dtype=torch.int32).cuda() * 3
    slots = torch.arange(T, dtype=torch.int32).cuda()

    def append(y):
        y = y.cuda()
        kc, vc, _, _ = new_pools(-(-T // 4), Hkv, 4, D, dt)
        q = attn.kv_append(y[:, :Hq], y[:, Hq: Hq + Hkv], y[:, Hq + Hkv:], slots, kc, vc, positions=pos,
                           cos=cos, sin=sin, interleaved=interleaved)
        back = [p.transpose(1, 2).reshape(-1, Hkv, D)[:T] for p in (kc, vc)]
        return torch.cat([q] + back, 1).cpu()

    got, want = append(x), append(plain)
    assert torch.equal(bits(got[..., :R]), bits(want[..., :R])) or R == 0     # rotated ones as without them
    kept, held = got[..., R:], x[..., R:]
    nan = torch.isnan(held)
    assert torch.equal(torch.isnan(kept), nan)
    assert torch.equal(bits(kept)[~nan], bits(held)[~nan])


# ---- value scales of any size ------------------------------------------------------


def check_rows(attn, prob, window=0):
    """Every row of an 8-bit problem against float64, with bounds from what the row itself sees.

    With weights w_j = p_j vs_j (p the softmax over the row's positions) and vbar = sum p_j |v_j|: a
    probability is off by 2 ds + (n + 8) 2^-22 and its weight by one rounding to fp16, 2^-11, where that is
    not below fp16's normal numbers, else by 2^-33 of the row's largest weight, times a code of up to
    448; scales under 2^-92 count as 2^-92 there, which leaves 2^-125 times 448 a position."""
    q, kc, vc, table, lens, ks, vs = prob
    out, lse = attn.paged_attention(q, kc, vc, table, lens, k_scale=ks, v_scale=vs, window=window, return_lse=True)
    Q, K, V, S, KS = np64(q), np64(kc), np64(vc), np64(vs), np64(ks)
    o, l, tab = np64(out), np64(lse), table.cpu().numpy()
    B, T, Hq, D = Q.shape
    ps, G = K.shape[2], Hq // K.shape[1]
    for b in range(B):
        n = int(lens[b])
        for t in range(T):
            at = np.arange(max(0, n - T + t + 1 - window) if window else 0, n - T + t + 1)
            page, slot = tab[b, at // ps], at % ps
            for h in range(Hq):
                hk = h // G
                key = K[page, hk, slot] * KS[page, hk, slot][:, None]
                code, scale = V[page, hk, slot], S[page, hk, slot]
                s = key @ Q[b, t, h] * D ** -0.5
                p = np.exp(s - s.max())
                total = p.sum()
                ref = (p * scale) @ code / total
                ds = (D + 8) * 2.0 ** -22 * (np.abs(key) @ np.abs(Q[b, t, h])).max() * D ** -0.5
                rel = 2 * ds + (len(at) + 8) * 2.0 ** -22 + 2.0 ** -11
                bound = (p * scale) @ np.abs(code) / total * rel
                bound += len(at) * 448 * (2.0 ** -33 * (p * scale).max() / total + 2.0 ** -125)
                err = np.abs(o[b, t, h] - ref)
                assert (err <= bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)).all(), (b, t, h, err.max())
                want = s.max() + math.log(total)
                assert abs(l[b, t, h] - want) <= ds + len(at) * 2.0 ** -22 + 2.0 ** -21 * (1 + abs(want))
    return out, lse


def scale_problem(D, T, Hq, lens, seed):
    return attn_problem(len(lens), T, Hq, 2, D, 16, lens, F8, seed=seed, nan=False)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sizes", [[1e-36], [2.0 ** -126], [0.0], [2.0 ** -105], [0.0, 2.0 ** -105, 0.01],
                                   [1e-36, 2.0 ** -100, 1e-20, 1e-5, 1.0], [1e-30, 1e12], [2.0 ** -105, 2.0 ** 60]],
                         ids=str)
def test_attention_value_scales_of_any_size(attn, sizes, D):
    """Scales all tiny, all zero, or tiny, zero and ordinary ones mixed, one token and drafts."""
    for T, Hq in ((1, 8), (3, 24)):
        prob = scale_problem(D, T, Hq, [300, 5, 40], seed=40 + T)
        g = torch.Generator().manual_seed(7)
        pick = torch.randint(0, len(sizes), prob[6].shape, generator=g)
        prob[6][:] = torch.tensor(sizes)[pick].cuda() * (0.5 + torch.rand(pick.shape, generator=g).cuda())
        check_rows(attn, prob)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 35, 2.0 ** 45, 2.0 ** 100])
def test_attention_unseen_large_scale_stays_out(attn, size, D):
    """A later draft token's large finite scale does not reach the rows before it, nor what a window has
    left behind the rows after it."""
    T, n = 4, 50
    prob = scale_problem(D, T, 8, [n], seed=50)
    kw = dict(k_scale=prob[5], v_scale=prob[6], return_lse=True)
    good, lg = attn.paged_attention(*prob[:5], **kw)
    prob[6][int(prob[3][0, (n - 1) // 16]), :, (n - 1) % 16] *= size
    bad, lb = check_rows(attn, prob)
    assert (np.abs(np64(bad[:, :3]) - np64(good[:, :3])) <= 2.0 ** -7 * np.abs(np64(good[:, :3])) + 1e-4).all()
    assert torch.allclose(lb, lg, rtol=0, atol=1e-5)
    prob = scale_problem(D, T, 8, [n], seed=51)
    prob[6][int(prob[3][0, 0]), :, 10] *= size       # inside the first row's window (n - 4 - 36 = 10) only
    check_rows(attn, prob, window=37)


def test_attention_improbable_large_value(attn):
    """A row's own position with a large scale and no weight in the softmax leaves the others their
    precision: score -90, scale 2^70 times theirs."""
    q, kc, vc, table, lens, ks, vs = scale_problem(64, 1, 2, [200], seed=52)
    q[:] = 1.0
    page = int(table[0, 3])
    kc.view(torch.uint8)[page, :, 5] = torch.full((2, 64), -1.0, device="cuda").to(F8).view(torch.uint8)
    ks[page, :, 5] = 90 / 8.0                        # 64 places of -90 / 8, times 1 / 8
    vs[page, :, 5] *= 2.0 ** 70
    check_rows(attn, (q, kc, vc, table, lens, ks, vs))


# ---- scores of any size ---------------------------------------------------------------


@pytest.mark.parametrize("size", [1e4, 1e9, 1e12, 1e20])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pdt", [BF, F8, F32], ids=["bf16", "fp8", "f32"])
def test_attention_huge_scores_are_one_hot(attn, pdt, D, size):
    """Finite scores so large that one position has all the weight: the output is its value (rounded to 16 bits
    at most twice, as a weight and as the result), whatever the size."""
    q, kc, vc, table, lens, ks, vs = attn_problem(3, 2, 6, 2, D, 16, [400, 37, 2], pdt, seed=60)
    q *= size
    out, lse = attn.paged_attention(q, kc, vc, table, lens, k_scale=ks, v_scale=vs, return_lse=True)
    o, l, Q, tab, found = np64(out), np64(lse), np64(q), table.cpu().numpy(), 0
    for b in range(3):
        for t in range(2):
            n = int(lens[b]) - 2 + t + 1
            at = np.arange(n)
            page, slot = tab[b, at // 16], at % 16
            for h in range(6):
                k, v = (np64(p)[page, h // 3, slot] for p in (kc, vc))
                if ks is not None:
                    k, v = (x * np64(s)[page, h // 3, slot][:, None] for x, s in ((k, ks), (v, vs)))
                s = k @ Q[b, t, h] * D ** -0.5
                smax = (np.abs(k) @ np.abs(Q[b, t, h])).max() * D ** -0.5
                order = np.argsort(s)
                # the runner-up is out of reach of the scores' rounding, and its weight below 2^-58
                if n > 1 and s[order[-1]] - s[order[-2]] < 2 * (D + 8) * 2.0 ** -22 * smax + 40:
                    continue
                found += 1
                want = v[order[-1]]
                assert (np.abs(o[b, t, h] - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -40).all(), (b, t, h)
                assert abs(l[b, t, h] - s[order[-1]]) <= (D + 8) * 2.0 ** -22 * smax + 1e-5
    assert found > 20


@pytest.mark.parametrize("D", [64, 128])
def test_attention_largest_queries_over_codes(attn, D):
    """Queries in the topmost binade of bf16 against small keys: ordinary scores."""
    q, kc, vc, table, lens, ks, vs = attn_problem(2, 1, 4, 2, D, 16, [100, 7], F8, seed=61)
    q *= 2.0 ** 126 / float(q.abs().max())
    q[0, 0, 1] *= 1.9
    q[0, 0, 2] *= 2 ** -126
    for i in range(2):
        q[i, 0, 0, 3], q[i, 0, 3, 5] = 2.0 ** 127 * 1.5, -2.0 ** 127 * 1.5
    ks *= 2.0 ** -125
    check_attn(attn, (q, kc, vc, table, lens, ks, vs), F8)


# ---- codes ---------------------------------------------------------------------------------


@pytest.mark.parametrize("T,Hq,Hkv,D,dt", [(70, 8, 4, 64, BF), (300, 8, 8, 128, BF), (200, 8, 8, 64, F32),
                                           (1300, 16, 8, 128, BF)])
def test_append_codes_are_the_quotient_rounded_once(attn, T, Hq, Hkv, D, dt):
    """Without norm and rotation, scale = max(amax, 2^-96) (1 / 448) and code = x / scale rounded to nearest
    even are bit for bit torch's: bf16 rows often hold quotients next to a tie (wherever 448 x / amax
    ends between two codes), which an inexact quotient sends either way."""
    g = torch.Generator().manual_seed(T)
    x = (torch.randn(T, Hq + 2 * Hkv, D, generator=g) * 2).to(BF).to(dt).cuda()
    x[1] *= 1e-33
    x[2] *= 2.0 ** 100
    x[3] = 0
    kc, vc, ks, vs = new_pools(-(-T // 16), Hkv, 16, D, F8)
    slots = torch.arange(T, dtype=torch.int32).cuda()
    attn.kv_append(x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:], slots, kc, vc, k_scale=ks, v_scale=vs)
    for pool, scale, rows in ((kc, ks, x[:, Hq: Hq + Hkv]), (vc, vs, x[:, Hq + Hkv:])):
        size = rows.float().abs().amax(-1).clamp(min=2.0 ** -96) * (1 / 448)
        codes = (rows.float() / size[..., None]).clamp(-448, 448).to(F8)
        got = pool.view(torch.uint8).transpose(1, 2).reshape(-1, Hkv, D)[:T]
        assert torch.equal(scale.transpose(1, 2).reshape(-1, Hkv)[:T], size)
        apart = (got != codes.view(torch.uint8)).sum()
        assert apart == 0, int(apart)
