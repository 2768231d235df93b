"""Which results of the 4-bit attention calls count as overlapping: views that share bytes are refused, views side by side
in one buffer are not (with CPU tensors, whose calls end behind those checks)."""
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.test_kv4_cpu import extend, outcome

N, H = 5, 16


def rows_and_lse_in_one_buffer(after):
    """[5][16] rows of 128 bf16 and, `after` bytes behind each row's start, a float: views of one buffer."""
    raw = torch.zeros(N * H * 512 + 512, dtype=torch.uint8)
    rows = raw[:N * H * 512].view(torch.bfloat16).view(N, H, 256)[..., :128]
    return rows, raw.view(torch.float32)[after // 4:].as_strided((N, H), (H * 128, 128))


@pytest.mark.parametrize("which", ["q", "out"])
@pytest.mark.parametrize("after,meet", [(0, True), (100, True), (252, True), (256, False), (300, False), (508, False), (512, True)])
def test_lse_between_the_rows(which, after, meet):
    rows, lse = rows_and_lse_in_one_buffer(after)
    got = outcome(extend, {which: rows, "lse": lse})
    assert ("lse overlaps q or out" in got[1]) == meet and got[2] != hpc.HPC_OK


@pytest.mark.parametrize("at,meet", [(0, True), (64, True), (120, True), (128, False), (136, True), (256, True)])
def test_q_and_out_in_one_buffer(at, meet):
    buf = torch.zeros(N * H * 256 + 256 * 2, dtype=torch.bfloat16)
    q = buf.as_strided((N, H, 128), (H * 256, 256, 1))
    out = buf[at:].as_strided((N, H, 128), (H * 256, 256, 1))
    assert ("out overlaps q" in outcome(extend, dict(q=q, out=out))[1]) == meet
