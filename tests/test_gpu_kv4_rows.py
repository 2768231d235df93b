"""One new token over a 4-bit cache: the 8 query rows of a KV head are independent, whatever their sizes. The rows'
results are compared with the 64-bit reference at the bounds that kv4_util.attend derives."""
import math

import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.kv4_util import Paged, cu_of, decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


@pytest.mark.parametrize("power", [40, 70, -70])
@pytest.mark.parametrize("hkv", [1, 3])
def test_rows_of_very_different_sizes(hkv, power):
    c = Paged([300, 70, 1], hkv=hkv, q_rows=3, seed=41, q_scale=6.0, ks=0.5)
    some = torch.rand(c.q.shape[:2], generator=torch.Generator().manual_seed(1)) < 0.3
    c.q[some] = c.q[some] * 2.0 ** power
    c.check(*decode(c, 1), cu_of([1] * 3))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_row_that_is_not_finite_spoils_no_other(value):
    c = Paged([500, 129, 9000], hkv=2, q_rows=3, seed=42)
    good, lse = decode(c, 1)
    finite = c.q.clone()
    rows = ((0, 0), (1, 11), (2, 7))
    for b, h in rows:
        c.q[b, h, 5] = value
    out, l2 = decode(c, 1)
    for b, h in rows:
        assert torch.isnan(out[b, h]).all() and not math.isfinite(l2[b, h].item())
        out[b, h], l2[b, h] = good[b, h], lse[b, h]
    c.q = finite
    c.check(out, l2, cu_of([1] * 3))
