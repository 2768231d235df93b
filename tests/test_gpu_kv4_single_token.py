"""Strides that no second token, or sequence, is reached by: any number may stand there, as a view of one row has it. And one
row of q for all new tokens (stride 0)."""
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.kv4_util import Paged, decode
from tests.test_gpu_kv4_extend import extend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


@pytest.mark.parametrize("stride", [0, 3, 1001, 1 << 42])
def test_one_new_token(stride):
    c = Paged([300], hkv=1, q_rows=1, seed=3)
    d = c.device()
    want, lse = extend(c, [1], d)
    for call in (lambda q, o, l: extend(c, [1], d, q=q, out=o, lse=l), lambda q, o, l: decode(c, 1, dict(d, q=q), out=o, lse=l)):
        q, out = (x.as_strided((1, 8, 128), (stride, 128, 1)) for x in (d["q"], torch.zeros_like(d["q"])))
        got, l2 = call(q, out, torch.zeros(8, device="cuda").as_strided((1, 8), (stride, 1)))
        c.check(got, l2, [0, 1])
    c.check(want, lse, [0, 1])


@pytest.mark.parametrize("stride", [0, 3, 1 << 42])
def test_one_sequence_of_new_tokens(stride):
    c = Paged([300], hkv=1, q_rows=3, seed=4)
    d = c.device()
    out = torch.zeros_like(d["q"])
    views = [x.as_strided((1, 3, 8, 128), (stride, 1024, 128, 1)) for x in (d["q"], out)]
    decode(c, 3, dict(d, q=views[0]), out=views[1])
    want, lse = decode(c, 3, d)
    assert torch.equal(out.view(want.shape), want)


def test_one_row_of_q_for_all_new_tokens():
    new = [20, 40]
    c = Paged([90, 40], hkv=2, q_rows=60, seed=5)
    c.q[:] = c.q[:1].clone()
    d = c.device()
    want, lse = extend(c, new, d)
    got, l2 = extend(c, new, d, q=d["q"][:1].expand(60, 16, 128))
    assert torch.equal(got, want) and torch.equal(l2, lse)
    c.check(want, lse, [0, 20, 60])
