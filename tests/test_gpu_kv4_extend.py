"""hpc_extend_kv4_attn against its definition in 64 bits; tolerances from kv4_util.attend (no states in f16 here)."""
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.kv4_util import Paged, cu_of, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


def extend(c, new, d=None, out=None, lse=None, scale=None, bits=0, q=None):
    d = d or c.device()
    shape = c.q.shape
    out = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full(shape[:-1], float("nan"), device="cuda") if lse is None else lse
    err = i32([0])
    hpc.hpc_extend_kv4_attn(d["q"] if q is None else q, d["k"], d["v"], d["bt"], d["sl"], i32(cu_of(new)), out, lse, softmax_scale=scale,
                            device_error=err, k_scale=c.ks, v_scale=c.vs)
    assert err.item() == bits
    return out, lse


BATCHES = {
    "one token": ([1], [0]),
    "edges": ([1, 15, 16, 17, 31, 32, 33, 64, 65], [0, 0, 1, 63, 64, 65, 127, 128, 0]),
    "none among them": ([0, 40, 0, 7, 0], [90, 0, 0, 1000, 64]),
    "prompt": ([512], [0]),
    "over a context": ([100, 3], [3000, 1]),
    "decode shape": ([1] * 20, [50 * i for i in range(20)]),
}


@pytest.mark.parametrize("hkv", [1, 2, 8])
@pytest.mark.parametrize("name", BATCHES)
def test_parity(name, hkv):
    new, old = BATCHES[name]
    c = Paged([n + o for n, o in zip(new, old)], hkv=hkv, q_rows=sum(new), seed=hkv)
    c.check(*extend(c, new), cu_of(new))


def test_both_cta_shapes_at_large_sizes():
    """Enough rows for two query tiles a CTA, and few enough for one, of the same sequences."""
    new, old = [150, 700, 33], [500, 100, 0]
    c = Paged([n + o for n, o in zip(new, old)], hkv=8, q_rows=sum(new), seed=3)
    out, lse = extend(c, new)
    c.check(out, lse, cu_of(new))
    few = Paged([n + o for n, o in zip(new, old)], hkv=1, q_rows=sum(new), seed=4)
    few.check(*extend(few, new), cu_of(new))


@pytest.mark.parametrize("scale,q_scale", [(0.5, 1.0), (None, 20.0), (None, 2.0 ** -110)])
def test_scales(scale, q_scale):
    new, old = [70, 20], [130, 7]
    c = Paged([n + o for n, o in zip(new, old)], hkv=2, q_rows=90, seed=5, q_scale=q_scale)
    c.check(*extend(c, new, scale=scale), cu_of(new), **({"scale": scale} if scale else {}))


def test_same_bits_and_strides():
    new, old = [45, 16, 1], [100, 0, 63]
    c = Paged([n + o for n, o in zip(new, old)], hkv=2, q_rows=62, seed=6)
    d = c.device()
    out, lse = extend(c, new, d)
    both = torch.stack([d["k"], d["v"]])
    o2, l2 = extend(c, new, dict(d, k=both[0], v=both[1]))
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    heads = dict(d, k=d["k"].transpose(0, 1).contiguous().transpose(0, 1), v=d["v"].transpose(0, 1).contiguous().transpose(0, 1))
    o2, l2 = extend(c, new, heads)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    wide = torch.full((64, 18, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(62, 16, 256, dtype=torch.bfloat16, device="cuda")
    q[..., 128:] = d["q"]
    extend(c, new, d, out=wide[1:63, 1:17, :128], q=q[..., 128:])
    assert torch.equal(wide[1:63, 1:17, :128], out)
    wide[1:63, 1:17, :128] = 5.0
    assert (wide == 5).all()


def test_rows_that_cannot_be():
    """More new tokens than positions, rows past the end of q, bad blocks: bits, and rows left as they were."""
    c = Paged([100, 50, 80], hkv=1, q_rows=60, seed=7)
    d = c.device()
    out, lse = extend(c, [20, 20, 20], d)
    sl = d["sl"].clone()
    sl[1] = 10
    o2, l2 = extend(c, [20, 20, 20], dict(d, sl=sl), bits=1)
    assert torch.equal(o2[:20], out[:20]) and torch.equal(o2[40:], out[40:]) and torch.isnan(o2[20:40]).all()
    o2, l2 = extend(c, [20, 20, 30], d, bits=1)
    assert torch.equal(o2[:40], out[:40]) and torch.isnan(o2[40:]).all() and torch.isnan(l2[40:]).all()
    bt = d["bt"].clone()
    bt[0, 0] = c.blocks
    o2, l2 = extend(c, [20, 20, 20], dict(d, bt=bt), bits=2)
    for r in c.rows[0]:
        r[:64] = 0
    c.check(o2, l2, cu_of([20, 20, 20]))


def test_graph():
    new, old = [40, 9], [70, 0]
    c = Paged([n + o for n, o in zip(new, old)], hkv=2, q_rows=49, seed=8)
    d = c.device()
    cu = i32(cu_of(new))
    out, lse = extend(c, new, d)
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hpc.hpc_extend_kv4_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], cu, o2, l2, k_scale=c.ks, v_scale=c.vs)
    graph.replay()
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_no_tokens():
    q = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, 1, 64, 72, dtype=torch.uint8, device="cuda")
    hpc.hpc_extend_kv4_attn(q, k, k, i32([[0]]), i32([0]), i32([0, 0]), q.clone())
