"""One new token over an e4m3 cache: query heads that share a KV head are independent, whatever their sizes, on every path
that decodes on mma.sync. Against the fp64 oracle at the parity tolerances."""
import numpy as np
import pytest
import torch

import oracle
import paged_gqa_decode_hpc_gb300 as hpc
from paged_gqa_decode_hpc_gb300 import workloads as W
from tests.gpu_util import assert_parity, device_workload, run_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


def step(w):
    d = device_workload(w)
    plan = hpc.hpc_decode_plan_create(w.q.shape[0], hpc.hpc_device_sm_count(), w.q.shape[1])
    out = torch.full(w.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(w.q.shape[:2], float("nan"), device="cuda")
    hpc.hpc_decode_step(d["q"], d["k"], d["v"], d["bt"], d["sl"], plan, hpc.hpc_device_sm_count(), out, lse,
                        k_scale=w.k_scale, v_scale=w.v_scale)
    assert hpc.hpc_decode_plan_status(plan) == 0
    plan.destroy()
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def shared_prefix(w):
    """One group that shares no block: its sequences' tiles are walked by warps."""
    d = device_workload(w)
    plan = hpc.hpc_decode_prefix_plan_create(w.q.shape[0], 1, hpc.hpc_device_sm_count(), w.q.shape[1])
    out = torch.full(w.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(w.q.shape[:2], float("nan"), device="cuda")
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    hpc.hpc_decode_prefix_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], none, plan, out, lse,
                               k_scale=w.k_scale, v_scale=w.v_scale)
    assert hpc.hpc_decode_plan_status(plan) == 0
    plan.destroy()
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


PATHS = {"step": step, "plan and attention": run_cuda, "static": lambda w: run_cuda(w, plan="static"), "shared prefix": shared_prefix}


def work(hkv=2):
    return W.make_workload(W.Config(96, "rows", 8 * hkv, hkv, "fp8_e4m3"), lengths=[300, 70, 1, 2000], seed=7)


@pytest.mark.parametrize("path", PATHS)
def test_small_rows_beside_huge_ones(path):
    """Rows of ordinary size beside one of 2^40 times it: the ordinary ones match the oracle."""
    w = work()
    ref_out, ref_lse = oracle.decode_workload(w)
    w.q[:, 3] = w.q[:, 3] * 2.0 ** 40
    out, lse = PATHS[path](w)
    keep = np.array([h for h in range(w.q.shape[1]) if h != 3])
    assert_parity(out[:, keep], lse[:, keep], ref_out[:, keep], ref_lse[:, keep], label=path)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("path", PATHS)
def test_a_row_that_is_not_finite_spoils_no_other(path, value):
    w = work()
    ref_out, ref_lse = oracle.decode_workload(w)
    w.q[0, 0, 5], w.q[3, 12, 9] = value, value
    out, lse = PATHS[path](w)
    keep = np.ones(w.q.shape[:2], dtype=bool)
    keep[0, 0] = keep[3, 12] = False
    assert_parity(out[keep], lse[keep], ref_out[keep], ref_lse[keep], label=path)
