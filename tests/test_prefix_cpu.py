"""Refusals of hpc_decode_prefix_attn and its plan that need no GPU: every tensor
is checked before anything touches a device, and the plan after the tensors."""
import math

import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc

I, U = hpc.HPC_ERR_INVALID_ARG, hpc.HPC_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    hpc.build()
    hpc.load_library()


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _i(*s):
    return torch.zeros(*s, dtype=torch.int32)


class NoPlan:
    handle = None


def _args(b=3, hkv=2, t=1):
    q = _bf(b, 8 * hkv, 128) if t == 1 else _bf(b, t, 8 * hkv, 128)
    return dict(q=q, k_cache=_bf(4, hkv, 64, 128), v_cache=_bf(4, hkv, 64, 128), block_table=_i(b, 5),
                seq_lens=_i(b), prefix_lens=_i(1), plan=NoPlan(), out=torch.zeros_like(q),
                lse=torch.zeros(q.shape[:-1]))


def _refused(args, **change):
    with pytest.raises(hpc.HpcError) as e:
        hpc.hpc_decode_prefix_attn(**{**args, **change}, stream=0)
    return e.value.status, str(e.value)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), I), (dict(q=torch.zeros(3, 16, 128)), I), (dict(q=_bf(3, 12, 128), out=_bf(3, 12, 128)), U),
    (dict(q=_bf(3, 16, 64), out=_bf(3, 16, 64)), U), (dict(out=_bf(3, 8, 128)), I), (dict(out=None), I),
    (dict(v_cache=_bf(5, 2, 64, 128)), I), (dict(k_cache=_bf(4, 2, 32, 128), v_cache=_bf(4, 2, 32, 128)), U),
    (dict(block_table=_i(2, 5)), I), (dict(block_table=_i(5, 3).t()), I), (dict(seq_lens=_i(4)), I),
    (dict(seq_lens=_i(6)[::2]), I), (dict(lse=torch.zeros(3, 8)), I), (dict(lse=_bf(3, 16)), I),
    (dict(prefix_lens=None), I), (dict(prefix_lens=_i(0)), I), (dict(prefix_lens=_i(2)), I),
    (dict(prefix_lens=torch.zeros(1)), I), (dict(prefix_lens=_i(2), cu_groups=_i(2)), I),
    (dict(prefix_lens=_i(4)[::2], cu_groups=_i(3)), I), (dict(cu_groups=torch.zeros(2)), I),
    (dict(prefix_lens=_i(4097), cu_groups=_i(4098)), I), (dict(softmax_scale=math.nan), I),
    (dict(softmax_scale=math.inf), I)])
def test_tensors(change, status):
    assert _refused(_args(), **change)[0] == status


def test_several_tokens():
    a = _args(t=2)
    assert _refused(a, q=_bf(3, 4, 16, 128)[:, :2])[0] == I  # tokens not evenly spaced over the batch
    assert "evenly spaced" in hpc.hpc_last_error()
    assert _refused(_args(t=9))[0] == U
    assert _refused(a, lse=torch.zeros(3, 16))[0] == I


def test_e4m3_scales():
    c = torch.zeros(4, 2, 64, 128, dtype=torch.uint8)
    assert _refused(_args(), k_cache=c, v_cache=c.clone(), k_scale=math.inf)[0] == I


def test_the_plan_comes_last():
    status, text = _refused(_args())
    assert status == I and "hpc_decode_prefix_plan_create" in text


@pytest.mark.parametrize("args,status", [
    ((0, 1, 152, 64), I), ((4, 1, 0, 64), I), ((4, 1, 152, 0), I), ((4, 1, 152, 12), I), ((4, 0, 152, 64), U),
    ((4, 9, 152, 64), U), ((4097, 1, 152, 64), U), ((4, 1, 152, 520), U), ((4, 1, 65537, 64), U)])
def test_plan_creation(args, status):
    with pytest.raises(hpc.HpcError) as e:
        hpc.hpc_decode_prefix_plan_create(*args)
    assert e.value.status == status
