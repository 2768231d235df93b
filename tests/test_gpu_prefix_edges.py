"""hpc_decode_prefix_attn at the ends of what its contract allows, against the fp64 decode oracle; inputs and
tolerances as in test_gpu_prefix.py, which derives them."""
import math

import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.test_gpu_prefix import SHAPES, Case

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


@pytest.mark.parametrize("q_len", [1, 2])
@pytest.mark.parametrize("fp8", [False, True])
def test_the_longest_sequence(fp8, q_len):
    """2^31 - 1 positions, all but the last 63 of them in one block: scores 0, V of -1, 0 and 1, so that the sums of a
    CTA, below 2^24, are exact. Of the last block slot 63 is behind the end (its K is NaN), and slot 62 hidden from the
    first of two new tokens. The merge rounds 2^31 and its like to 24 bits, a few times."""
    n, tiles = 2 ** 31 - 1, 2 ** 25
    g = torch.Generator().manual_seed(1)
    k, v = torch.zeros(2, 1, 64, 128), torch.zeros(2, 1, 64, 128)
    v[0] = torch.randint(-1, 2, (1, 64, 128), generator=g)
    k[1, 0, 63] = v[1, 0, 63] = float("nan")
    k, v = (x.cuda().to(torch.float8_e4m3fn if fp8 else torch.bfloat16) for x in (k, v))
    table = torch.zeros(1, tiles, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    shape = (1, 8, 128) if q_len == 1 else (1, q_len, 8, 128)
    q = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(shape[:-1], device="cuda")
    i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
    plan = hpc.hpc_decode_prefix_plan_create(1, q_len, hpc.hpc_device_sm_count(), 8)
    hpc.hpc_decode_prefix_attn(q, k, v, table, i32(n), i32(0), plan, out, lse)
    assert hpc.hpc_decode_plan_status(plan) == 0
    total = v[0, 0].double().sum(0) * (tiles - 1)
    for t in range(q_len):
        ref = total / (n - (q_len - 1 - t))
        got = out.view(q_len, 8, 128)[t].double()
        assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20).all()
        assert ((lse.view(q_len, 8)[t].double() - math.log(n)).abs() <= 2.0 ** -18).all()


@pytest.mark.parametrize("captured", [False, True])
def test_different_steps_queued_on_one_plan(captured):
    """Steps of different sizes, types and prefixes one after the other on one plan, nothing waited for in between (or
    one graph of them all, replayed): each has the bits that it has alone."""
    plan = hpc.hpc_decode_prefix_plan_create(80, 4, 152, 64)
    steps = []
    for name, hkv, q_len, fp8 in (("three tiles", 8, 1, False), ("two", 1, 4, True), ("groups", 2, 3, False), ("long", 1, 1, False),
                                  ("one sequence", 8, 1, True), ("short and empty", 4, 2, False), ("33 pairs", 2, 1, True),
                                  ("no prefix", 1, 1, False), ("long", 8, 2, True), ("17 pairs", 1, 1, False)):
        groups = [(p, [n + (q_len if n else 0) for n in lens]) for p, lens in SHAPES[name]]
        c = Case(groups, hkv=hkv, q_len=q_len, fp8=fp8, seed=21)
        d = c.device()
        alone = c.run(d, plan=plan)
        c.check(alone)
        steps.append((c, d, alone, [torch.empty_like(x) for x in alone]))

    def queue(order):
        for i in order:
            c, d, _, (out, lse) = steps[i]
            hpc.hpc_decode_prefix_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], d["pl"], plan, out, lse, cu_groups=d["cu"],
                                       k_scale=c.scales[0], v_scale=c.scales[1])
    orders = [torch.randperm(len(steps), generator=torch.Generator().manual_seed(i)).tolist() for i in range(30)]
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for order in orders:
                queue(order)
    for _ in range(10 if captured else 1):
        for _, _, _, got in steps:
            for x in got:
                x.fill_(float("nan"))
        torch.cuda.synchronize()
        if captured:
            graph.replay()
        else:
            for order in orders:
                queue(order)
        assert hpc.hpc_decode_plan_status(plan) == 0
        for _, _, alone, got in steps:
            assert all(torch.equal(a, b) for a, b in zip(alone, got))
