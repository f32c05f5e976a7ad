"""The cache's write where a warp takes several passes: from 2432 warps on, up to four passes of 512 places a warp
(two with fp32 rows and with 4-bit pools of heads of 64), spread evenly.  Definitions and bounds are
test_kv_forms_gpu.py's."""
import pytest
import torch

from test_attn_forms_gpu import F4, IDS
from test_attn_gpu import BF, F8, F32, attn  # noqa: F401
from test_kv_forms_gpu import DEALT, check_append

pytestmark = pytest.mark.gpu

# (R of D, interleaved, sections of R / 2, axes): a whole head in half pairs, a part in adjacent ones, not at
# all; the same with axes
TURNS = [(1, False, None, 1), (2, True, None, 1), (0, False, None, 1),
         (1, False, lambda n: (1,) * n, 3), (2, True, lambda n: (n // 2, n - n // 2), 2)]


@pytest.mark.parametrize("turn", range(len(TURNS)))
@pytest.mark.parametrize("dt,pdt", [(BF, BF), (BF, F8), (BF, F4), (F32, F32), (F32, F8), (F32, F4)],
                         ids=lambda t: IDS[t])
@pytest.mark.parametrize("passes", [3, 4])
@pytest.mark.parametrize("D", [64, 128])
def test_appends_of_several_passes_a_warp(attn, D, passes, dt, pdt, turn):
    part, interleaved, sections, axes = TURNS[turn]
    R = D // part if part else 0
    per = 512 // D                                   # rows of a pass
    Hq, Hkv = (per // 2, per // 2) if passes == 3 else (2 * per - per // 2, per // 2)
    case = (2437, Hq, Hkv, D, R, interleaved, turn % 2 == 0, 16, dt, pdt, sections and sections(R // 2), axes)
    check_append(attn, case, pad=[(0, -1), (2436, 2 ** 31 - 1), (1217, -5)])


@pytest.mark.parametrize("pdt", [BF, F8, F4], ids=lambda t: IDS[t])
@pytest.mark.parametrize("dt", [BF, F32], ids=lambda t: IDS[t])
def test_appends_of_several_warps_a_token(attn, dt, pdt):
    """12 passes of a token: three warps of four, six of two."""
    if dt == F32 and pdt == BF:
        pdt = F32
    check_append(attn, (820, 32, 8, 128, 128, False, True, 64, dt, pdt, None, 1))
    check_append(attn, (820, 32, 8, 128, 128, False, True, 64, dt, pdt, DEALT, 3), token_major=True)
