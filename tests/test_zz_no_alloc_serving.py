"""The serving operators allocate nothing (a plan takes all of its own when it is created): the first call of every size
can be captured, which an allocation would end, and no call changes the device's free memory. Collected late on
purpose, like the allocation-free entry's tests; torch's own allocator only serves the buffers made beforehand."""
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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(seqs, tokens):
    """append of `tokens` new tokens for each of `seqs` sequences, and the truncate that undoes it."""
    width = -(-tokens // 64)
    n = seqs * width
    lens, new, zero = _i32([0] * seqs), _i32([tokens] * seqs), _i32([0] * seqs)
    free, count, table = torch.arange(n, dtype=torch.int32, device="cuda"), _i32([n]), _i32([[-1] * width] * seqs)
    cu, pos, slots = _i32([0] * (seqs + 1)), _i32([0] * (seqs * tokens)), _i32([0] * (seqs * tokens))

    def call():
        hpc.hpc_block_table_append(lens, new, free, count, n, table, lens, cu, pos, slots, count)
        hpc.hpc_block_table_truncate(lens, zero, table, n, free, count, lens, count)
    return call


def _rope(tokens, hkv, fp8, norm, **kw):
    rows = [torch.zeros(tokens, h, 128, dtype=torch.bfloat16, device="cuda") for h in (8 * hkv, hkv, hkv)]
    t = torch.uint8 if fp8 else torch.bfloat16
    caches = [torch.zeros(-(-tokens // 64), hkv, 64, 128, dtype=t, device="cuda") for _ in range(2)]
    q8 = torch.zeros(tokens, 8 * hkv, 128, dtype=torch.uint8, device="cuda") if fp8 else None
    at, w = torch.arange(tokens, dtype=torch.int32, device="cuda"), torch.ones(128, device="cuda") if norm else None
    table = hpc.hpc_rope_init(**kw)
    return lambda: hpc.hpc_rope_kv_write(*rows, at, at, table, rows[0], *caches, q_norm_weight=w, k_norm_weight=w, q_out_fp8=q8)


def _prefix(groups, q_len, hkv, fp8, sms=152):
    c = Case([(p, [n + q_len for n in lens]) for p, lens in groups], q_len=q_len, hkv=hkv, fp8=fp8)
    d, plan = c.device(), hpc.hpc_decode_prefix_plan_create(len(c.lens), q_len, sms, 8 * hkv)
    out, lse = torch.empty_like(d["q"]), torch.empty(d["q"].shape[:-1], device="cuda")
    return lambda: hpc.hpc_decode_prefix_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], d["pl"], plan, out, lse, cu_groups=d["cu"],
                                              k_scale=c.scales[0], v_scale=c.scales[1])


def test_free_memory_stays():
    calls = [_tables(3, 70), _tables(200, 500)]
    for norm in (False, True):
        for kw in (dict(), dict(rot_dim=90), dict(interleaved=True, rot_dim=64)):
            calls += [_rope(n, hkv, fp8, norm, **kw) for n, hkv, fp8 in ((5, 1, False), (3000, 8, True))]
    for q_len in (1, 4):
        for fp8 in (False, True):
            calls += [_prefix([(128, [150, 190])], q_len, 1, fp8), _prefix([(2000, [2100] * 40), (0, [900] * 10)], q_len, 8, fp8),
                      _prefix([(700, [701] * 20)], q_len, 8, fp8), _prefix([(700, [701] * 9)], q_len, 4, fp8)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="global"):
        for call in calls:
            call()
    graph.replay()
    for call in calls:
        call()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    for call in calls[::-1] + calls:
        call()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == before
