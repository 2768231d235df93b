"""cu_q_lens that cannot be: a sequence whose rows would leave q sets HPC_DEVCHK_BAD_LENGTH and takes nothing from the
others, whose rows are written with the same bits; its own are left as they were."""
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.kv4_util import Paged, cu_of, i32

pytestmark = pytest.mark.gpu
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


def run(c, d, cu):
    out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c.q.shape[:2], float("nan"), device="cuda")
    err = i32([0])
    hpc.hpc_extend_kv4_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], i32(cu), out, lse, device_error=err, k_scale=c.ks, v_scale=c.vs)
    return out, lse, err.item()


# sequences 0, 1, 2 (and empty ones behind them): which rows are still written
@pytest.mark.parametrize("cu,kept", [
    ([0, 20, 1000000, 1000020], [(0, 20)]), ([0, 20, 61, 81], [(0, 20)]), ([0, 20, 40, 1000000], [(0, 20), (20, 40)]),
    ([0, 20, TOP, TOP], [(0, 20)]), ([0, 20, TOP - 8, TOP], [(0, 20)]), ([-5, 20, 40, 60], [(20, 40), (40, 60)]),
    ([0, TOP, 0, TOP - 31], []), ([-2 ** 31, 20, 40, 60], [(20, 40), (40, 60)]), ([0, 20, 40, 60], [(0, 20), (20, 40), (40, 60)])])
@pytest.mark.parametrize("empty", [0, 40])
@pytest.mark.parametrize("hkv", [1, 64])
def test_a_sequence_that_leaves_q_takes_nothing_from_others(cu, kept, empty, hkv):
    c = Paged([100, 50, 80] + [0] * empty, hkv=hkv, q_rows=60, seed=7)
    d = c.device()
    good, lse, bits = run(c, d, cu_of([20, 20, 20] + [0] * empty))
    assert bits == 0
    out, l2, bits = run(c, d, cu + [cu[-1]] * empty)
    assert bits == (0 if len(kept) == 3 else 1)
    left = torch.ones(60, dtype=torch.bool, device="cuda")
    for a, z in kept:
        left[a:z] = False
    assert torch.isnan(out[left]).all() and torch.isnan(l2[left]).all()
    assert torch.equal(out[~left], good[~left]) and torch.equal(l2[~left], lse[~left])
