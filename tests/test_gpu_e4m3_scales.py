"""E4m3 K scales that are not positive numbers of fp32's normal range, on the tensor-core kernels, against the fp64
oracle at the parity tolerances: a cache of zeros may have scale 0, and the header admits every finite scale."""
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from paged_gqa_decode_hpc_gb300 import workloads as W
from tests import test_gpu_decode_tc as tc
from tests import test_gpu_extend as ext
from tests.gpu_util import assert_parity

pytestmark = pytest.mark.gpu

SCALES = [0.0, -0.0, 1e-44, -1e-44, -0.02]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


@pytest.mark.parametrize("k_scale", SCALES)
@pytest.mark.parametrize("q_len", [3, 8])
def test_multi_token_decode(k_scale, q_len):
    w = W.make_workload(tc._cfg(16, 2, True), lengths=[9, 64, 130, 701], seed=q_len)
    w.k_scale = k_scale
    q = W.make_multi_query(w, q_len, seed=3)
    ref_out, ref_lse = tc._oracle(w, q)
    out, lse = tc.run(w, q)
    assert_parity(out, lse, ref_out, ref_lse, label=f"k_scale {k_scale}, q_len {q_len}")


@pytest.mark.parametrize("k_scale", SCALES)
@pytest.mark.parametrize("tiles", [1, 2])
def test_extend(k_scale, tiles):
    w = W.make_workload(ext._cfg(16, 2, True), lengths=[70, 9, 130, 701], seed=5)
    w.k_scale = k_scale
    q, cu = W.make_extend_query(w, [70, 3, 66, 17], seed=6)
    ref_out, ref_lse = ext._oracle(w, q, cu)
    out, lse = ext.run_extend(w, q, cu, tpc=tiles)
    assert_parity(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref_out, ref_lse,
                  label=f"k_scale {k_scale}, {tiles} query tiles a CTA")
