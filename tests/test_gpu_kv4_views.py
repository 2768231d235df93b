"""q, out and lse of a step as views of one buffer: side by side they are served, with the bits that separate tensors give;
where they share bytes they are refused."""
import itertools
import random

import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.kv4_util import Paged, decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


@pytest.mark.parametrize("q_len", [1, 2, 5])
@pytest.mark.parametrize("pad", [0, 1])
def test_side_by_side_with_padded_tokens(q_len, pad):
    """Heads of q, then heads of out, in every token's row of a buffer whose sequences hold `pad` tokens more."""
    c = Paged([200, 65, 900], hkv=2, q_rows=3 * q_len, seed=43)
    d = c.device()
    want, lse = decode(c, q_len, d)
    buf = torch.full((3, q_len + pad, 33, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    q, out = buf[:, :q_len, :16, :128], buf[:, :q_len, 16:32, :128]
    q.copy_(d["q"].view(3, q_len, 16, 128))
    if q_len == 1:
        q, out = q[:, 0], out[:, 0]
    got, l2 = decode(c, q_len, dict(d, q=q), out=out)
    assert torch.equal(got, want) and torch.equal(l2, lse)
    out.fill_(5.0)
    q.fill_(5.0)
    assert (buf == 5).all()


def places(shape, strides, at, size):
    """The bytes of a view's pieces of `size` bytes (shape and strides in bytes of its outer dimensions)."""
    got = []
    for i in itertools.product(*(range(n) for n in shape)):
        a = at + sum(x * y for x, y in zip(i, strides))
        got += range(a, a + size)
    return got


def test_exactly_the_views_that_share_bytes_are_refused():
    """Random views of one buffer with q's, out's (and lse's) sequences and heads at the same strides, checked byte for
    byte. What is refused is refused on the host; what is served stays inside the buffer."""
    rng = random.Random(5)
    c = Paged([70, 3], hkv=1, q_rows=4, seed=44)
    d = c.device()
    plan = hpc.hpc_decode_kv4_plan_create(2, 2, hpc.hpc_device_sm_count(), 8)
    buf = torch.zeros(1 << 16, dtype=torch.bfloat16, device="cuda")
    floats = buf.view(torch.float32)
    seen = {True: 0, False: 0}
    for _ in range(400):
        order = rng.sample(["b", "t", "h"], 3)
        size, extent, strides = {"b": 2, "t": 2, "h": 8}, 128 + 8 * rng.randint(0, 20), {}
        for x in order:
            strides[x] = extent + 8 * rng.choice([0, 0, 1, 17])
            extent = strides[x] * size[x]
        st = (strides["b"], strides["t"], strides["h"], 1)
        span = sum((size[x] - 1) * strides[x] for x in size) + 128
        assert 3 * span < buf.numel()
        at = rng.choice([8 * rng.randint(0, span // 8), 128, 8 * (strides["h"] // 8 - 16)] + [v - 128 for v in strides.values()])
        q, out = buf.as_strided((2, 2, 8, 128), st), buf[max(at, 0):].as_strided((2, 2, 8, 128), st)
        la = max(at, 0) // 2 + rng.choice([-2, 64, 65, 66])
        inside = la >= 0 and rng.random() < 0.5 and all(v % 2 == 0 for v in strides.values())
        lse = floats[la:].as_strided((2, 2, 8), tuple(v // 2 for v in st[:3])) if inside else torch.zeros(2, 2, 8, device="cuda")
        outer = [(2, 2, 8), tuple(2 * v for v in st[:3])]
        views = [places(*outer, 0, 256), places(*outer, 2 * max(at, 0), 256)] + ([places(*outer, 4 * la, 4)] if inside else [])
        own = [len(set(v)) == len(v) for v in views]
        meet = not all(own) or len(set().union(*map(set, views))) != sum(map(len, views))
        seen[meet] += 1
        if meet:
            with pytest.raises(hpc.HpcError, match="overlap"):
                hpc.hpc_decode_kv4_attn(q, d["k"], d["v"], d["bt"], d["sl"], plan, out, lse)
        else:
            hpc.hpc_decode_kv4_attn(q, d["k"], d["v"], d["bt"], d["sl"], plan, out, lse)
    assert hpc.hpc_decode_plan_status(plan) == 0 and min(seen.values()) > 40
