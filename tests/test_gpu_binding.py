"""The same outputs through the extension module and through ctypes, on the
current stream, a given one and the default one."""
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.test_gpu_prefix import Case as Prefix
from tests.test_gpu_rope import Case as Rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()
    assert hpc._native is not None


def both(monkeypatch, run):
    fast = run()
    with monkeypatch.context() as m:
        m.setattr(hpc, "_native", None)
        plain = run()
    assert len(fast) == len(plain)
    for a, b in zip(fast, plain):
        assert torch.equal(a.cpu(), b.cpu())
    return fast


@pytest.mark.parametrize("fp8", [False, True])
def test_rope(monkeypatch, fp8):
    c = Rope(50, 16, 2, normed=True, fp8=fp8, q_fp8=fp8, token_major=fp8, seed=21)

    def run():
        q, q8, caches = c.run()
        return [q, *caches] + ([q8] if fp8 else [])
    both(monkeypatch, run)


@pytest.mark.parametrize("q_len,fp8", [(1, False), (3, True)])
def test_prefix(monkeypatch, q_len, fp8):
    c = Prefix([(256, [300, 290, 700]), (64, [65, 80])], q_len=q_len, fp8=fp8, seed=22)
    c.check(both(monkeypatch, lambda: c.run()))
    both(monkeypatch, lambda: c.run(scale=0.05, stream=torch.cuda.Stream()))


@pytest.mark.parametrize("stream", ["current", "given", "default"])
def test_tables(monkeypatch, stream):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")

    def run():
        t = dict(lens=i32([10, 64, 0]), new=i32([60, 1, 130]), free=i32(list(range(20))), count=i32([20]),
                 table=i32([[30] * 4, [31] * 4, [32] * 4]), cu=i32([9] * 4), pos=i32([9] * 200), slots=i32([9] * 200),
                 err=i32([0]))
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        kw = {"current": {}, "given": {"stream": s}, "default": {"stream": 0}}[stream]
        hpc.hpc_block_table_append(t["lens"], t["new"], t["free"], t["count"], 40, t["table"], t["lens"], t["cu"],
                                   t["pos"], t["slots"], t["count"], device_error=t["err"], **kw)
        torch.cuda.synchronize()
        grown = [t[k].clone() for k in ("lens", "count", "table", "cu", "pos", "slots")]
        hpc.hpc_block_table_truncate(t["lens"], i32([10, 64, 0]), t["table"], 40, t["free"], t["count"], t["lens"],
                                     t["count"], device_error=t["err"], **kw)
        torch.cuda.synchronize()
        assert t["count"].item() == 20 and t["lens"].tolist() == [10, 64, 0] and t["err"].item() == 0
        return grown + [t["free"]]
    got = both(monkeypatch, run)
    assert got[0].tolist() == [70, 65, 130] and got[1].item() == 20 - 1 - 1 - 3
