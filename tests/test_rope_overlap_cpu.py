"""Outputs of hpc_rope_kv_write that share memory with its inputs or each other: refused, and views that lie side by
side in one buffer are not. Without a GPU an accepted call ends at the first question to the device."""
import random

import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc

D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if torch.cuda.is_available():
        pytest.skip("an accepted call would run on these host buffers")
    hpc.build()
    hpc.load_library()


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _call(q_in, k_in, v_in, q_out, q_out_fp8=None, k_cache=None, v_cache=None):
    n, hkv = q_in.shape[0], k_in.shape[1]
    k_cache, v_cache = (_bf(2, hkv, 64, D) if c is None else c for c in (k_cache, v_cache))
    z = torch.zeros(n, dtype=torch.int32)
    with pytest.raises(hpc.HpcError) as e:
        hpc.hpc_rope_kv_write(q_in, k_in, v_in, z, z.clone(), hpc.hpc_rope_init(), q_out, k_cache, v_cache,
                              q_out_fp8=q_out_fp8, stream=0)
    return e.value.status, str(e.value)


def refused(*a, **kw):
    status, text = _call(*a, **kw)
    assert status in (hpc.HPC_ERR_INVALID_ARG, hpc.HPC_ERR_CUDA), text
    if status == hpc.HPC_ERR_INVALID_ARG:
        assert "overlap" in text
    return status == hpc.HPC_ERR_INVALID_ARG


def _fused(n, hq, hkv, extra=0):
    x = _bf(n, hq + 2 * hkv + extra, D)
    return x, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]


@pytest.mark.parametrize("n,hq,hkv", [(1, 8, 1), (5, 16, 2), (300, 64, 8)])
def test_views_of_one_buffer(n, hq, hkv):
    x, q, k, v = _fused(n, hq, hkv, extra=2 * hq)
    rest = x[:, hq + 2 * hkv:]
    assert not refused(q, k, v, _bf(n, hq, D))
    assert not refused(q, k, v, q)                    # in place
    assert not refused(q, k, v, rest[:, :hq])         # a place of its own in the same rows
    fp8 = torch.zeros(n, hq, D, dtype=torch.uint8)
    assert not refused(q, k, v, q, fp8)
    assert refused(q, k, v, x[:, 1:hq + 1])           # a head later
    assert refused(q, k, v, x[:, 2 * hkv:hq + 2 * hkv])  # on k and v, at its end
    if n > 1:
        assert refused(q[:-1], k[:-1], v[:-1], q[1:])    # a token later
        assert refused(q, k, v, _bf(1, hq, D).expand(n, hq, D))
        assert refused(q, k, v, _bf(n, 1, D).expand(n, hq, D))
    b = rest.contiguous().view(torch.uint8)            # [n][2 hq][256 bytes]
    row = b.view(n, -1)
    bf, e4 = row[:, :hq * 2 * D].view(torch.bfloat16).view(n, hq, D), row[:, hq * 2 * D:hq * 3 * D].view(n, hq, D)
    assert not refused(bf, k, v, bf, e4)
    assert refused(q, k, v, bf, row[:, 2 * D:2 * D + hq * D].view(n, hq, D))
    assert refused(bf, k, v, _bf(n, hq, D), row[:, :hq * D].view(n, hq, D))


def test_k_and_v_are_not_outputs():
    _, q, k, v = _fused(4, 8, 8)
    assert refused(q, k, v, k) and refused(q, k, v, v)
    assert refused(q, k, v, q, q_out_fp8=k.view(torch.uint8)[..., :D])


def test_caches_are_not_outputs():
    _, q, k, v = _fused(4, 8, 1)
    x = _bf(2 * 64 * D * 2 + 4 * 8 * D)
    cache, rest = x[:2 * 64 * D].view(2, 1, 64, D), x[2 * 64 * D:]
    assert not refused(q, k, v, rest[:4 * 8 * D].view(4, 8, D), k_cache=cache)
    assert refused(q, k, v, x[2 * 64 * D - 8:][:4 * 8 * D].view(4, 8, D), k_cache=cache)
    e4 = x[64 * D:][:4 * 4 * D].view(torch.uint8).view(4, 8, D)
    assert refused(q, k, v, q, q_out_fp8=e4, v_cache=cache) and not refused(q, k, v, q, q_out_fp8=e4)


def test_against_all_pairs_of_rows():
    """Strided views at random places of one buffer: refused exactly if two rows share bytes."""
    rng = random.Random(1)
    seen = [0, 0]
    for _ in range(3000):
        n, hq = rng.choice([1, 2, 3, 5]), rng.choice([1, 2, 3])
        sn, sh = (rng.choice([8, 64, 128, 136, 256, 384, 520, 640, 1024]) for _ in range(2))
        size = 8000
        x = _bf(size)

        def view(heads):
            top = size - ((n - 1) * sn + (heads - 1) * sh + D)
            return rng.randrange(0, max(1, min(top, rng.choice([64, 600, top]))) // 8 + 1) * 8

        places = [view(hq), view(hq)]
        if (max(places) + (n - 1) * sn + (hq - 1) * sh + D) > size:
            continue
        q_in, q_out = (x.as_strided((n, hq, D), (sn, sh, 1), p) for p in places)
        rows = [[p + i * sn + h * sh for i in range(n) for h in range(hq)] for p in places]
        itself = any(abs(a - b) < D for i, a in enumerate(rows[1]) for b in rows[1][:i])
        cross = places[0] != places[1] and any(abs(a - b) < D for a in rows[0] for b in rows[1])
        want = itself or cross
        assert refused(q_in, _bf(n, hq, D), _bf(n, hq, D), q_out) == want, (n, hq, sn, sh, places)
        seen[want] += 1
    assert min(seen) > 300
