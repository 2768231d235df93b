"""The serving loop of test_gpu_serving_run.py with the bounds that the attention's own tests derive: with an e4m3
cache probabilities are rounded to f16, 2^-11 of each and 2^-25 of the largest at least, not to bf16."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests import test_gpu_serving_run as run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


@pytest.mark.parametrize("q_len", [1, 3])
def test_a_serving_loop_on_e4m3(q_len, monkeypatch):
    checked = []

    def check_attention(self, out, lse, q, counts):
        ref, ref_lse, size = self.reference(q, counts)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.all(np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + (2 * 2.0 ** -11 + 2.0 ** -14) * size)
        assert np.all(np.abs(lse - ref_lse) <= 2.0 ** -14 + 2.0 ** -22 * np.abs(ref_lse))
        checked.append(len(ref))
    monkeypatch.setattr(run.Server, "check_attention", check_attention)
    run.test_a_serving_loop(True, q_len)
    assert len(checked) == 4
