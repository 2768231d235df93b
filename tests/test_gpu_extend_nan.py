"""Extend attention over keys that are not numbers: out and lse of the rows that see one are NaN (lse is -inf only where a
row sees no position), all other rows keep their bits."""
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from paged_gqa_decode_hpc_gb300 import workloads as W
from tests import test_gpu_extend as ext
from tests.kv4_util import Paged, cu_of
from tests.test_gpu_kv4_extend import extend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


def compare(out, lse, good, good_lse, spoilt):
    assert torch.isnan(out[spoilt]).all() and torch.isnan(lse[spoilt]).all()
    assert torch.equal(out[~spoilt], good[~spoilt]) and torch.equal(lse[~spoilt], good_lse[~spoilt])


# (KV heads, new tokens): one query tile a CTA, whose keys two chains share, and two
@pytest.mark.parametrize("hkv,new", [(1, [20, 40]), (2, [1, 16]), (8, [330, 40])])
@pytest.mark.parametrize("at", [3, 64 + 5, 2 * 64 + 63, 300])
def test_4_bit_rows(hkv, new, at):
    c = Paged([n + 290 for n in new], hkv=hkv, q_rows=sum(new), seed=at)
    good, lse = extend(c, new)
    if at >= c.lens[0]:
        at = c.lens[0] - 1
    c.k[c.table[0, at // 64].long(), hkv - 1, at % 64, 64 + at % 8] = 0x7F
    out, l2 = extend(c, new)
    spoilt = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    spoilt[max(at - 290, 0):new[0], 8 * (hkv - 1):] = True  # token t sees positions up to 290 + t
    compare(out, l2, good, lse, spoilt)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("hkv,new", [(1, [20, 40]), (8, [330, 40])])
def test_4_bit_a_row_of_q(hkv, new, value):
    """The other rows stay within the bounds that kv4_util.attend derives (a row's size may choose between two roundings
    for the rows of its warp)."""
    c = Paged([n + 100 for n in new], hkv=hkv, q_rows=sum(new), seed=4)
    good, lse = extend(c, new)
    finite = c.q.clone()
    c.q[17, 5, 9] = value
    out, l2 = extend(c, new)
    assert torch.isnan(out[17, 5]).all() and torch.isnan(l2[17, 5])
    out[17, 5], l2[17, 5] = good[17, 5], lse[17, 5]
    c.q = finite
    c.check(out, l2, cu_of(new))


@pytest.mark.parametrize("tiles", [1, 2])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("at", [3, 64 + 5, 300])
def test_wider_rows(fp8, tiles, at):
    w = W.make_workload(ext._cfg(16, 2, fp8), lengths=[330, 300], seed=at)
    new = [40, 21]
    q, cu = W.make_extend_query(w, new, seed=6)
    good, lse = ext.run_extend(w, q, cu, tpc=tiles)
    k = w.k_cache.clone()
    bits = k.view(torch.uint8 if fp8 else torch.int16)
    bits[int(w.block_table[0, at // 64]), 1, at % 64, 77] = 0x7F if fp8 else 0x7FC0
    out, l2 = ext.run_extend(w, q, cu, k=k.cuda(), tpc=tiles)
    spoilt = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    spoilt[max(at - 290, 0):40, 8:] = True
    compare(out, l2, good, lse, spoilt)
