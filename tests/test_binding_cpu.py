"""The extension module behind the calls of a few microseconds (csrc/binding.cpp)
and the ctypes path that it stands beside: the same refusals, word for word, and
the ctypes path for whatever the module does not take. Nothing reaches a device."""
import ctypes

import numpy as np
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc


@pytest.fixture(scope="module", autouse=True)
def _lib():
    hpc.build()
    hpc.load_library()
    if hpc._native is None:
        pytest.skip("built without Python's headers")


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _b(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def append(**kw):
    a = dict(seq_lens=_i(3), new_lens=_i(3), free_blocks=_i(8), free_count=_i(1), num_blocks=8, block_table=_i(3, 4),
             seq_lens_out=_i(3), cu_q_lens=_i(4), positions=_i(5), slots=_i(5), free_count_out=_i(1), stream=0)
    return hpc.hpc_block_table_append(**{**a, **kw})


def truncate(**kw):
    a = dict(seq_lens=_i(3), to_lens=_i(3), block_table=_i(3, 4), num_blocks=8, free_blocks=_i(8), free_count=_i(1),
             seq_lens_out=_i(3), free_count_out=_i(1), stream=0)
    return hpc.hpc_block_table_truncate(**{**a, **kw})


def rope(**kw):
    a = dict(q_in=_b(2, 8, 128), k_in=_b(2, 1, 128), v_in=_b(2, 1, 128), positions=_i(2), slots=_i(2),
             rope=hpc.hpc_rope_init(), q_out=_b(2, 8, 128), k_cache=_b(3, 1, 64, 128), v_cache=_b(3, 1, 64, 128), stream=0)
    return hpc.hpc_rope_kv_write(**{**a, **kw})


class NoPlan:
    handle = None


def prefix(**kw):
    a = dict(q=_b(2, 8, 128), k_cache=_b(3, 1, 64, 128), v_cache=_b(3, 1, 64, 128), block_table=_i(2, 2), seq_lens=_i(2),
             prefix_lens=_i(1), plan=NoPlan(), out=_b(2, 8, 128), lse=torch.zeros(2, 8), stream=0)
    return hpc.hpc_decode_prefix_attn(**{**a, **kw})


class Odd:
    """Not a tensor: what a tensor is asked for, wrong."""
    dtype, shape = torch.int32, [3]

    def data_ptr(self):
        raise ValueError("no storage")

    def dim(self):
        return 1

    def stride(self):
        return (1,)


def outcome(call, kw):
    try:
        call(**kw)
    except Exception as e:  # noqa: BLE001 (what it is, is compared)
        return type(e), str(e), getattr(e, "status", None)
    return None


BAD = [
    (append, dict(new_lens=_i(2))), (append, dict(free_count=_i(2))), (append, dict(num_blocks=-1)),
    (append, dict(block_table=_i(3))), (append, dict(positions=torch.zeros(5))), (append, dict(slots=torch.zeros(5).double())),
    (append, dict(seq_lens=_i(1, 1, 1, 1, 1))), (append, dict(seq_lens=Odd())), (append, dict(seq_lens=3)),
    (append, dict(num_blocks="8")), (append, dict(num_blocks=2**31 - 1)), (append, dict(cu_q_lens=None)),
    (append, dict(device_error=5)), (append, dict(stream="s")),
    (truncate, dict(to_lens=_i(3).float())), (truncate, dict(free_blocks=_i(2, 4))), (truncate, dict(num_blocks=2.5e9)),
    (truncate, dict(seq_lens=None)), (truncate, dict(block_table=_i(3, 4).t())),
    (rope, dict(q_in=_b(2, 8, 64))), (rope, dict(eps=-1.0)), (rope, dict(eps="x")), (rope, dict(rope=None)),
    (rope, dict(rope=hpc.HpcRope())), (rope, dict(rope=b"table")), (rope, dict(k_cache=_i(3, 1, 64, 128))),
    (rope, dict(q_out_fp8=torch.zeros(2, 8, 128, dtype=torch.uint8), q_fp8_scale=0.0)),
    (rope, dict(v_in=Odd())), (rope, dict(q_norm_weight=_b(64))),
    (prefix, dict()), (prefix, dict(q=_b(2, 8, 64))), (prefix, dict(prefix_lens=_i(2))), (prefix, dict(lse=_i(2, 8))),
    (prefix, dict(softmax_scale=float("nan"))), (prefix, dict(softmax_scale="1")), (prefix, dict(k_scale=None)),
    (prefix, dict(out=torch.zeros(2, 8, 128).half())), (prefix, dict(seq_lens=_i(2)[::2])),
]


@pytest.mark.parametrize("n", range(len(BAD)))
def test_both_paths_refuse_alike(n, monkeypatch):
    call, kw = BAD[n]
    native = outcome(call, kw)
    monkeypatch.setattr(hpc, "_native", None)
    plain = outcome(call, kw)
    assert native is not None and native == plain


def test_arguments_that_only_the_plain_path_takes():
    """A list for a shape, a number that is no int: None, and nothing has been called."""
    n = hpc._native
    assert n.append(*[None] * 4, 8, *[None] * 8) is not None  # all null: the entry refuses that
    assert n.append(*[None] * 13) is None                     # no number of blocks
    assert n.append(1, 2) is None
    assert n.truncate(*[Odd()] * 10) is None
    assert n.rope_kv_write(*[3.5] * 18) is None
    assert n.prefix_attn(*["q"] * 14) is None


def test_references_are_returned():
    import sys
    t = _i(3)
    kw = dict(new_lens=t, free_count=_i(2))
    before = sys.getrefcount(t), sys.getrefcount(torch.int32), sys.getrefcount(t.shape)
    for _ in range(1000):
        outcome(append, kw)
    after = sys.getrefcount(t), sys.getrefcount(torch.int32), sys.getrefcount(t.shape)
    assert all(abs(a - b) < 20 for a, b in zip(before, after))


def test_numbers_of_other_types():
    assert outcome(append, dict(num_blocks=np.int64(-1))) == outcome(append, dict(num_blocks=-1))
    assert outcome(rope, dict(eps=np.float32(-1))) == outcome(rope, dict(eps=-1.0))
    assert outcome(prefix, dict(softmax_scale=torch.tensor(float("inf")))) == outcome(prefix, dict(softmax_scale=float("inf")))
    assert ctypes.sizeof(hpc.HpcRope) == 12 + 2 * 64 * 4
