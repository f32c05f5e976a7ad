"""Pieces of prompts and batches of many rows over bf16 pools: what the kernels carry from one item, one
launch and one call to the next.  References and bounds are test_attn_forms_gpu.py's."""
import pytest
import torch

from test_attn_forms_gpu import BF, check, problem
from test_attn_gpu import attn  # noqa: F401

pytestmark = pytest.mark.gpu


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
