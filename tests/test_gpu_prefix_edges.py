"""hpc_decode_prefix_attn at the ends of what its contract allows, against the fp64 decode oracle; inputs and
tolerances as in test_gpu_prefix.py, which derives them."""
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.test_gpu_prefix import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


@pytest.mark.parametrize("k_scale", [0.0, -0.0, 1e-44, -1e-44, -0.21])
@pytest.mark.parametrize("q_len", [1, 3, 8])
def test_e4m3_scales_that_are_not_positive(k_scale, q_len):
    # shared tiles of one and of two row tiles, own tiles masked at their ends; a cache of zeros may have scale 0
    c = Case([(192, [193 + q_len + 11 * i for i in range(4)]), (64, [70 + q_len + i for i in range(18)])], q_len=q_len,
             fp8=True, seed=q_len, q_scale=4.0)
    c.scales = (k_scale, 0.17)
    c.check()


def test_one_token_of_a_wider_batch():
    # q [B][1][H_q][128] whose sequences lie more than a token apart: evenly spaced all the same
    c = Case([(128, [200, 190, 130]), (0, [70])], seed=4)
    d, n = c.device(), len(c.lens)
    wide = torch.full((n, 4, 16, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    out, lse = (torch.full(s, 5.0, dtype=t, device="cuda") for s, t in (((n, 2, 16, 128), torch.bfloat16), ((n, 3, 16), torch.float32)))
    d["q"] = wide[:, 2:3].copy_(d["q"][:, None])
    c.run(d, out=out[:, :1], lse=lse[:, 1:2])
    c.check((out[:, 0], lse[:, 1]))
    assert (out[:, 1] == 5).all() and (lse[:, ::2] == 5).all()
