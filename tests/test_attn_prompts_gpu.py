"""Pieces of prompts and batches of many rows over bf16 pools: what the kernels carry from one item, one
launch and one call to the next.  References and bounds are test_attn_forms_gpu.py's."""
import ctypes
import itertools
import json
import os
import subprocess
import sys

import pytest
import torch

from test_attn_forms_gpu import BF, check, problem
from test_attn_gpu import attn  # noqa: F401

pytestmark = pytest.mark.gpu


def launches(attn, prob, **kw):
    """Kernels that a call launches: 1 where k_paged_prompt takes it, 2 where the others do, 3 where the lengths
    tell.  (Counted in a captured graph, which is not run.)"""
    q, pools, table, lens = prob
    B, T, Hq, D = q.shape
    need = attn.paged_attention_workspace_size(B, T, Hq, pools.Hkv, D, pools.pdt)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    call = lambda: attn.paged_attention(q, *pools.pools, table, lens, out=out, workspace=ws, **pools.kw, **kw)
    cuda = ctypes.CDLL("libcuda.so.1")
    s = torch.cuda.Stream()
    handle, graph, n = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p(), ctypes.c_size_t()
    with torch.cuda.stream(s):
        call()                                       # (what a first call sets up cannot be captured)
        s.synchronize()
        assert cuda.cuStreamBeginCapture_v2(handle, 2) == 0
        try:
            call()
        finally:
            assert cuda.cuStreamEndCapture(handle, ctypes.byref(graph)) == 0
    assert cuda.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0 and cuda.cuGraphDestroy(graph) == 0
    return n.value


@pytest.mark.parametrize("D", [64, 128])
def test_calls_whose_lengths_tell_follow_one_another(attn, D):
    """Equal and uneven batches of 40 sequences, which different kernels take, one after another without a
    wait over the same workspace and output; each result is copied by the next kernel on the stream."""
    B, T, Hq, Hkv = 40, 32, 32, 8
    longest = 6000
    q, pools, table, lens = problem(B, T, Hq, Hkv, D, 16, [longest] + [700] * (B - 1), BF, 71)
    kinds = [[700] * B, [longest] + [40] * (B - 1), [0] * B, [longest, 0] * 2 + [33] * (B - 4), [31, 32, 700, 1] * 10]
    kinds[3][2] = 0                                  # (only sequence 0 has pages for the longest)
    sets = [torch.tensor(k, dtype=torch.int32).cuda() for k in kinds]
    out = torch.empty_like(q)
    ws = torch.empty(max(attn.paged_attention_workspace_size(B, T, Hq, Hkv, D), 1), dtype=torch.uint8, device="cuda")
    call = lambda n, **kw: attn.paged_attention(q, *pools.pools, table, n, **kw)
    want = []
    for n in sets:
        want.append(call(n))
        torch.cuda.synchronize()
        check(attn, (q, pools, table, n))
    got = []
    for _ in range(4):
        for n in sets:
            call(n, out=out, workspace=ws)
            got.append(out.clone())
            out.fill_(7.0)
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % len(sets)]), i


@pytest.mark.parametrize("T,n", [(1300, 1400), (300, 1400)])
@pytest.mark.parametrize("D", [64, 128])
def test_log_sums_are_rounded_where_they_must_be(attn, D, T, n):
    """Large scores that rise from tile to tile, a little in most rows and by more than a reference may lag
    in one of four, so that all rows' references move with each tile.  Scores q0 600 + q1 k1 are exact in
    f32, and so is scale log2(e) up to f32's log2(e), so what a log sum errs by is

    * 2^-17 of its log2, and the rest: a weight's exponent is below 16 in size where it counts (2^-21), its
      exponential 2^-22, sums of 50 in turn 50 2^-24, log2 2^-22,
    * half a step of f32 of the log2 (reference plus log2 of the sum), and of the result."""
    Hq, Hkv, G, scale = 32, 8, 4, 0.5
    q, pools, table, lens = problem(1, T, Hq, Hkv, D, 16, [n], BF, 63)
    q.zero_()
    row = torch.arange(T, device="cuda")[:, None] * G + torch.arange(G, device="cuda")
    q0 = 1.25 + (row * 37 % 96) / 128
    q1 = torch.where(row % G == 0, 128.0, 1.0)
    j = torch.arange(n, device="cuda")
    k1 = (j // 128 * 8 + j * 5 % 8) / 64
    q[0, :, :, 0], q[0, :, :, 1] = q0.repeat(1, Hkv).to(BF), q1.repeat(1, Hkv).to(BF)
    keys = torch.zeros(n, D, device="cuda")
    keys[:, 0], keys[:, 1] = 600, k1
    pools.pools[0][table[0].long()[j // 16], :, j % 16] = keys[:, None].to(BF)
    assert torch.equal(keys.to(BF).float(), keys) and torch.equal(q0.to(BF).double(), q0.double())
    _, lse = attn.paged_attention(q, *pools.pools, table, lens, scale=scale, return_lse=True)
    log2e = float(torch.tensor(1.4426950408889634, dtype=torch.float32))
    for t0 in range(0, T, 100):
        t = slice(t0, t0 + 100)
        s = (600 * q0[t].double()[..., None] + q1[t].double()[..., None] * k1.double()) * (scale * log2e)
        own = n - T + torch.arange(T, device="cuda")[t]
        s = s.masked_fill(j > own[:, None, None], float("-inf"))
        top = s.amax(-1)
        log2 = top + torch.log2(torch.exp2(s - top[..., None]).sum(-1))
        ref = log2 * 0.6931471805599453
        half = lambda v: torch.exp2(torch.floor(torch.log2(v.abs())) - 24)
        bound = 0.6931471805599453 * (half(log2) + 2.0 ** -17) + half(ref) + 2.0 ** -19
        for h in range(Hkv):
            assert ((lse[0, t, h * G: (h + 1) * G].double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("T", [1300, 300])
@pytest.mark.parametrize("D", [64, 128])
def test_references_of_any_size_follow_one_another(attn, D, T):
    """Scores from -2^24 over -2^12 and 2^12 to 2^21, a size for 64 positions: a row's weight is that of the last
    size that it sees, shared by its positions.  Nothing but roundings to 16 bits (weight, result) and, in the
    log sums, of the factor of the scores."""
    Hq, Hkv, n = 32, 8, 1400
    q, pools, table, lens = problem(1, T, Hq, Hkv, D, 16, [n], BF, 64)
    j = torch.arange(n, device="cuda")
    size = j // 64
    key = torch.where(size < 13, -torch.exp2((12 - size).double()), torch.exp2((size - 13).double()))
    keys = torch.zeros(n, D, device="cuda", dtype=BF)
    keys[:, 5] = key.to(BF)
    pools.pools[0][table[0].long()[j // 16], :, j % 16] = keys[:, None]
    q.zero_()
    q[..., 5] = 2.0 ** 12
    out, lse = attn.paged_attention(q, *pools.pools, table, lens, scale=1.0, return_lse=True)
    own = n - T + torch.arange(T, device="cuda")
    score = torch.where(j <= own[:, None], key * 2.0 ** 12, -torch.inf)
    top = score.amax(1, keepdim=True)
    weight = (score == top).double()
    count = weight.sum(1, keepdim=True)
    v = pools.rows(1, table[0].long()[j // 16], j % 16)
    want, most = (torch.einsum("tj,jhd->thd", weight / count, x).repeat_interleave(Hq // Hkv, 1) for x in (v, v.abs()))
    assert ((out[0].double() - want).abs() <= 2.0 ** -7 * most + 1e-30).all()
    assert ((lse[0].double() - top - torch.log(count)).abs() <= 2.0 ** -20 * (1 + top.abs())).all()


# ---- layouts of the pools ------------------------------------------------------------------------

def in_order(x, order):
    """The pool x [pages, Hkv, ps, D] with its first three dimensions in memory in another order."""
    back = [order.index(i) for i in range(3)]
    return x.permute(*order, 3).contiguous().permute(*back, 3)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("order", list(itertools.permutations(range(3))), ids=str)
def test_pools_in_any_order_of_memory(attn, D, order):
    for Hkv in (8, 1):
        q, pools, table, lens = prob = problem(2, 500 if Hkv == 8 else 3000, 4 * Hkv, Hkv, D, 48, [700, 300], BF, 65)
        kw = dict(window=300, sinks=4)
        want, _ = check(attn, prob, **kw) if Hkv == 8 else (attn.paged_attention(q, *pools.pools, table, lens, **kw), 0)
        assert launches(attn, prob, **kw) == 1
        pools.pools = [in_order(x, order) for x in pools.pools]
        assert launches(attn, prob, **kw) == 1
        assert torch.equal(attn.paged_attention(q, *pools.pools, table, lens, **kw), want)


def test_pools_without_a_tensor_map(attn):
    """Heads that lie some places further apart than their tokens take, or on top of one another: served too."""
    q, pools, table, lens = prob = problem(1, 1300, 32, 8, 128, 16, [1400], BF, 66)
    pages = pools.pools[0].shape[0]
    assert launches(attn, prob) == 1
    wide = []
    for x in pools.pools:
        room = torch.zeros(pages, 8, 16 * 128 + 8, dtype=BF, device="cuda")
        room[..., : 16 * 128] = x.flatten(2)
        wide.append(room[..., : 16 * 128].unflatten(2, (16, 128)))
    pools.pools = wide
    assert not wide[0].is_contiguous() and launches(attn, prob) == 2
    check(attn, prob)
    check(attn, prob, 200, 3)
    # one page or one head whose stride is whatever it is
    q, pools, table, lens = prob = problem(1, 1300, 32, 8, 128, 1408, [1400], BF, 67)
    want, _ = check(attn, prob)
    pools.pools = [x[int(table[0, 0]):][:1].as_strided((1, 8, 1408, 128), (7, 1408 * 128, 128, 1)) for x in pools.pools]
    table.zero_()
    assert launches(attn, prob) == 1
    assert torch.equal(attn.paged_attention(q, *pools.pools, table, lens), want)


# ---- the path's own cases -----------------------------------------------------------------------

CASES = [
    # (T, Hq, Hkv, D, ps, lens, window, sinks): pages of 16 n and rows enough for the path
    (700, 16, 2, 128, 48, [2000], 300, 0),
    (700, 16, 2, 128, 48, [2000, 650], 300, 5),
    (300, 40, 8, 64, 16, [1700, 300, 301, 40], 129, 200),              # more sinks than a window
    (130, 8, 8, 128, 16, [130, 257, 128, 640, 129], 128, 1),           # one row behind a block
    (128, 8, 8, 128, 128, [128, 5000, 1, 127, 200, 129], 1, 1),        # a row sees itself and the sink
    (257, 6, 6, 64, 112, [257, 1300, 256, 255, 30, 4000, 1], 1000, 64),
    (130, 8, 8, 128, 16, [300] * 12, 0, 0),
    (1300, 32, 8, 128, 16, [3000, 0], 0, 0),                           # items without positions between others
    (1300, 32, 8, 64, 16, [0, 3000, 0], 900, 20),
    (700, 32, 8, 128, 32, [2000, 0, 0, 5, 0, 701], 0, 0),
    (700, 32, 8, 64, 32, [699, 0, 1400], 250, 0),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_cases_that_the_path_takes(attn, case):
    T, Hq, Hkv, D, ps, lens, window, sinks = case
    prob = problem(len(lens), T, Hq, Hkv, D, ps, lens, BF, 300 + T)
    assert launches(attn, prob, window=window, sinks=sinks) == 1
    check(attn, prob, window, sinks)


@pytest.mark.parametrize("ps", [16, 48, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_missing_pages(attn, D, ps):
    """Pages that are no pages, among those that rows see, at the sinks and between sinks and window; a length
    beyond the table."""
    q, pools, table, lens = prob = problem(4, 300, 32, 4, D, ps, [1700, 1000, 310, 600], BF, 14, poison=False)
    M = table.shape[1]
    table[0, 240 // ps: 640 // ps], table[0, 0], table[1, :] = -1, pools.pools[0].shape[0], -7
    table[3, 560 // ps], table[2, 1] = -1, 2 ** 31 - 1
    lens[2] = M * ps + 77
    for window, sinks in ((0, 0), (100, 50), (100, 1), (0, 9)):
        assert launches(attn, prob, window=window, sinks=sinks) == 1
        check(attn, prob, window, sinks)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 0), (200, 9)])
def test_unseen_values_stay_out_of_half_items(attn, D, bad, window, sinks):
    """All items are halved: an infinity or NaN in either half of a tile reaches the rows that see it alone."""
    T, Hq, Hkv, ps, n = 300, 32, 8, 16, 900
    q, pools, table, lens = prob = problem(1, T, Hq, Hkv, D, ps, [n], BF, 15)
    kw = dict(window=window, sinks=sinks)
    assert launches(attn, prob, **kw) == 1
    call = lambda: attn.paged_attention(q, *pools.pools, table, lens, **kw)
    good = call()
    e = n - T + torch.arange(T, device="cuda")
    G = Hq // Hkv
    for at in (0, 3, 100, 400, 460, 550, 640, 700, 767, 768, 898, 899):
        place = (int(table[0, at // ps]), 2, at % ps, 7)
        was = pools.pools[1][place].clone()
        pools.pools[1][place] = bad
        got = call()
        pools.pools[1][place] = was
        see = e >= at
        if window:
            see &= (at > e - window) | (at < sinks)
        hit = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
        hit[0, :, 2 * G: 3 * G, 7] = see[:, None]
        assert torch.equal(got[~hit], good[~hit])
        assert not torch.isfinite(got[hit]).any()


@pytest.mark.parametrize("B,T,longest", [(1, 1500, 3000), (2, 1300, 2500), (1, 300, 2000)])
def test_replays_match_the_definition(attn, B, T, longest):
    """One captured call, replayed with other lengths, each result against the definition."""
    q, pools, table, lens = prob = problem(B, T, 32, 8, 128, 16, [longest] * B, BF, 68, poison=False)
    kw = dict(window=700, sinks=9)
    assert launches(attn, prob, **kw) == 1
    out = torch.empty_like(q)
    ws = torch.empty(max(attn.paged_attention_workspace_size(B, T, 32, 8, 128), 1), dtype=torch.uint8, device="cuda")
    call = lambda: attn.paged_attention(q, *pools.pools, table, lens, out=out, workspace=ws, **kw)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in (longest - 1, T + 60, 200, 0, 1, longest):
        lens.fill_(n)
        lens[-1] = n if B == 1 else longest - n
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want, _ = check(attn, prob, 700, 9)
        assert torch.equal(got, want)


def test_calls_whose_lengths_tell_on_two_streams_and_in_one_graph(attn):
    """Two such calls at once, each with its own workspace; then both in a graph over one."""
    B, T, Hq, Hkv = 14, 32, 32, 8
    probs = [problem(B, T, Hq, Hkv, D, 16, n, BF, 80 + D) for D, n in ((64, [9000] + [40] * 13), (128, [1600] * 14))]
    for p in probs:
        assert launches(attn, p) == 3
    call = lambda p, **kw: attn.paged_attention(p[0], *p[1].pools, p[2], p[3], **kw)
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
    outs = [torch.empty_like(p[0]) for p in probs]
    ws = torch.empty(max(attn.paged_attention_workspace_size(B, T, Hq, Hkv, D) for D in (64, 128)), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            for p, out in zip(probs, outs):
                call(p, out=out, workspace=ws)
    for _ in range(3):
        for out in outs:
            out.fill_(7.0)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, x) for out, x in zip(outs, want))


DEBUG_CHILD = r"""
import ctypes, json, sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import test_attn_prompts_gpu as t
from state_space_model_gb300 import _native, attn
import torch
assert _native.LIB_PATH.endswith("libssd_gb300_debug.so"), _native.LIB_PATH
for case in t.CASES:
    T, Hq, Hkv, D, ps, lens, window, sinks = case
    t.check(attn, t.problem(len(lens), T, Hq, Hkv, D, ps, lens, t.BF, 300 + T), window, sinks)
for D in (64, 128):
    t.test_calls_whose_lengths_tell_follow_one_another(attn, D)
    t.test_missing_pages(attn, D, 48)
    for order in ((0, 2, 1), (1, 2, 0)):
        t.test_pools_in_any_order_of_memory(attn, D, order)
lib = _native.load()
st = lib.ssd_device_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
print(json.dumps({"status": st, "detail": lib.ssd_last_error_detail().decode()}))
"""


def test_debug_build_finds_every_index_in_bounds(attn):
    from state_space_model_gb300 import build
    build.build(debug_bounds=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", DEBUG_CHILD, root], env=dict(os.environ, SSD_DEBUG_BOUNDS="1"),
                       cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["status"] == 0, out["detail"]
