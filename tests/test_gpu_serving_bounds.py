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


@pytest.mark.parametrize("fp8", [False, True])
def test_one_captured_step_for_any_numbers_of_new_tokens(fp8):
    """append packs a step's tokens, the attention takes [B][q_len]: between them one gather by cu_q_lens, sequences'
    tokens at the right. Sequences with fewer tokens than q_len, with none, and finished ones (length 0) are one
    captured graph; rows before a sequence's own tokens mean nothing."""
    B, T, prefix = 5, 4, 100
    s = run.Server(fp8, B, 31)
    b = s.buffers(64)
    b["new"][0] = 64
    s.write(b)
    s.follow(b)
    s.table[1:4] = s.table[0]
    s.lens[1:4] = 64
    s.ref["table"] = [list(s.ref["table"][0]) if i < 4 else r for i, r in enumerate(s.ref["table"])]
    s.ref["lens"] = [64] * 4 + [0]
    new = [36, 36 + 80, 36 + 5, 36 + 27, 50]
    b = s.buffers(sum(new))
    b["new"].copy_(run._i32(new))
    s.write(b)
    s.follow(b)
    d = s.buffers(B * T)
    groups, prefixes, at = run._i32([0, 4, B]), run._i32([prefix, 0]), torch.arange(T, device="cuda")
    plan = hpc.hpc_decode_prefix_plan_create(B, T, hpc.hpc_device_sm_count(), run.HQ)
    out = torch.zeros(B, T, run.HQ, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(B, T, run.HQ, device="cuda")

    def step():
        s.write(d)
        rows = (d["cu"][1:, None] - T + at).clamp(0, B * T - 1)
        hpc.hpc_decode_prefix_attn(d["q"][rows], *s.caches, s.table, s.lens, prefixes, plan, out, lse, cu_groups=groups,
                                   k_scale=s.scales[0], v_scale=s.scales[1])
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()  # no new tokens yet: it only attends
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    assert hpc.hpc_decode_plan_status(plan) == 0
    for it, counts in enumerate(([4, 4, 4, 4, 4], [1, 4, 0, 3, 2], [0, 2, 4, 0, 1], [3, 0, 1, 1, 4], [0, 0, 0, 0, 0])):
        if it == 2:  # row 0 is done: its own blocks go back, the shared one stays with the others
            s.truncate([64] + s.ref["lens"][1:])
            s.lens[0] = s.ref["lens"][0] = 0
        if it == 3:  # the others shorten by their last draft
            s.truncate([max(0, n - 1) for n in s.ref["lens"]])
            counts = [0] + counts[1:]
        d["qkv"].copy_(torch.randn(d["qkv"].shape, generator=s.gen, device="cuda"))
        d["new"].copy_(run._i32(counts))
        graph.replay()
        torch.cuda.synchronize()
        assert hpc.hpc_decode_plan_status(plan) == 0
        s.follow(d)
        live = torch.tensor([[t >= T - c for t in range(T)] for c in counts])
        if sum(counts):
            s.check_attention(out[live], lse[live], d["q"][:sum(counts)], counts)
        for i, n in enumerate(s.ref["lens"]):
            if n == 0:
                assert (out[i] == 0).all() and (lse[i] == float("-inf")).all()
    s.check_cache()
