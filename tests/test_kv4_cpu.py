"""The 4-bit reference's pins, and the refusals of the 4-bit calls that need no GPU: every tensor is checked before
anything touches a device, by the extension module and by ctypes alike."""
import math

import numpy as np
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from oracle import kv4_ref

I, U = hpc.HPC_ERR_INVALID_ARG, hpc.HPC_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    hpc.build()
    hpc.load_library()


# ------------------------------------------------------------------ the reference
def test_e4m3_table():
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv4_ref.E4M3, want)


def test_nearest_against_brute_force():
    for table in (kv4_ref.E2M1, kv4_ref.E4M3):
        x = np.concatenate([table, (table[1:] + table[:-1]) / 2, np.linspace(0, table[-1] * 1.1, 999)])
        for v, i in zip(x, kv4_ref.nearest(x, table)):
            d = np.abs(table - v)
            best = np.flatnonzero(d == d.min())
            assert i == (best[0] if len(best) == 1 else best[best % 2 == 0][0])


def test_rows_by_hand():
    x = np.zeros((1, 128))
    x[0, :4] = [6.0, -2.5, 0.25, 5.0]   # scale 1: 6, -2 (a tie to even), 0 (a tie), 4 (a tie)
    x[0, 16] = 3000.0                   # past 448 * 6: saturates
    r = kv4_ref.rows(x, 1.0)
    assert r[0, :2].tolist() == [0x7 | 0xC0, 0x0 | 0x60] and r[0, 64:66].tolist() == [0x38, 0x7E]
    v = kv4_ref.values(r, 0.5)
    assert v[0, :4].tolist() == [3.0, -1.0, 0.0, 2.0] and v[0, 16] == 1344.0 and not v[0, 32:].any()


def test_round_trip_error():
    x = np.random.default_rng(0).normal(size=(200, 128))
    v = kv4_ref.values(kv4_ref.rows(x, 0.003), 0.003)
    top = np.abs(x).reshape(200, 8, 16).max(-1).repeat(16, -1)
    # a scale is off by at most 1/16 of itself, a code by 1 of 6 (above 4: half of 2)
    assert (np.abs(v - x) <= top * (1 + 1 / 16) / 6 + 1e-12).all()


# ------------------------------------------------------------------ refusals
def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _i(*s):
    return torch.zeros(*s, dtype=torch.int32)


def _c(*s):
    return torch.zeros(*s, dtype=torch.uint8)


class NoPlan:
    handle = None


def write(**kw):
    a = dict(q_in=_bf(2, 16, 128), k_in=_bf(2, 2, 128), v_in=_bf(2, 2, 128), positions=_i(2), slots=_i(2), rope=hpc.hpc_rope_init(),
             q_out=_bf(2, 16, 128), k_cache=_c(3, 2, 64, 72), v_cache=_c(3, 2, 64, 72), stream=0)
    return hpc.hpc_rope_kv4_write(**{**a, **kw})


def decode(**kw):
    a = dict(q=_bf(3, 16, 128), k_cache=_c(4, 2, 64, 72), v_cache=_c(4, 2, 64, 72), block_table=_i(3, 5), seq_lens=_i(3), plan=NoPlan(),
             out=_bf(3, 16, 128), lse=torch.zeros(3, 16), stream=0)
    return hpc.hpc_decode_kv4_attn(**{**a, **kw})


def extend(**kw):
    a = dict(q=_bf(5, 16, 128), k_cache=_c(4, 2, 64, 72), v_cache=_c(4, 2, 64, 72), block_table=_i(3, 5), seq_lens=_i(3), cu_q_lens=_i(4),
             out=_bf(5, 16, 128), lse=torch.zeros(5, 16), stream=0)
    return hpc.hpc_extend_kv4_attn(**{**a, **kw})


_buffer = _bf(8, 40, 128)
_kv = _c(3, 2, 2, 64, 72)
CACHES = [
    (dict(k_cache=_c(4, 2, 64, 128), v_cache=_c(4, 2, 64, 128)), U), (dict(k_cache=_c(4, 2, 32, 72), v_cache=_c(4, 2, 32, 72)), U),
    (dict(k_cache=_c(4, 2, 64, 80)[..., :72], v_cache=_c(4, 2, 64, 80)[..., :72]), U),
    (dict(k_cache=_c(4, 64, 2, 72).transpose(1, 2), v_cache=_c(4, 64, 2, 72).transpose(1, 2)), U),
    (dict(k_cache=_c(5, 2, 64, 72)), I), (dict(k_cache=_bf(4, 2, 64, 72), v_cache=_bf(4, 2, 64, 72)), I), (dict(k_cache=None), I),
    (dict(v_cache=_c(4, 2, 64 * 72)), I), (dict(k_scale=0.0), I), (dict(v_scale=-1.0), I), (dict(k_scale=math.nan), I),
    (dict(v_scale=math.inf), I), (dict(k_cache=_c(4 * 2 * 4608 + 8)[8:].view(4, 2, 64, 72)), I),
    (dict(k_cache=_c(4, 2, 4616)[..., :4608].unflatten(-1, (64, 72)), v_cache=_c(4, 2, 4616)[..., :4608].unflatten(-1, (64, 72))), I),
]
BAD = [(decode, kw, st) for kw, st in CACHES] + [(extend, kw, st) for kw, st in CACHES] + [
    (decode, dict(), I),  # the plan, last of all
    (decode, dict(q=None), I), (decode, dict(q=torch.zeros(3, 16, 128)), I), (decode, dict(q=_bf(3, 12, 128), out=_bf(3, 12, 128)), U),
    (decode, dict(q=_bf(3, 16, 64), out=_bf(3, 16, 64)), U), (decode, dict(q=_bf(3, 9, 16, 128), out=_bf(3, 9, 16, 128), lse=None), U),
    (decode, dict(q=_bf(3, 0, 16, 128), out=_bf(3, 0, 16, 128), lse=None), I), (decode, dict(out=_bf(3, 8, 128)), I), (decode, dict(out=None), I),
    (decode, dict(q=_bf(3, 16, 132)[..., :128]), I), (decode, dict(q=_bf(3 * 16 * 128 + 1)[1:].view(3, 16, 128)), I),
    (decode, dict(q=_bf(3, 128, 16).transpose(1, 2)), I), (decode, dict(block_table=_i(2, 5)), I), (decode, dict(block_table=_i(5, 3).t()), I),
    (decode, dict(seq_lens=_i(4)), I), (decode, dict(seq_lens=_i(6)[::2]), I), (decode, dict(seq_lens=_i(3).long()), I),
    (decode, dict(lse=torch.zeros(3, 8)), I), (decode, dict(lse=_bf(3, 16)), I), (decode, dict(softmax_scale=math.nan), I),
    (decode, dict(softmax_scale=math.inf), I), (decode, dict(softmax_scale="1"), None), (decode, dict(k_scale=None), None),
    (decode, dict(softmax_scale=1e30, k_scale=1e30), I),
    (extend, dict(q=None), I), (extend, dict(q=_bf(5, 12, 128), out=_bf(5, 12, 128)), U), (extend, dict(q=_bf(1, 5, 16, 128)), I),
    (extend, dict(out=_bf(4, 16, 128)), I), (extend, dict(lse=torch.zeros(5, 8)), I), (extend, dict(cu_q_lens=_i(3)), I),
    (extend, dict(cu_q_lens=None), I), (extend, dict(cu_q_lens=_i(8)[::2]), I), (extend, dict(cu_q_lens=_i(0)), I),
    (extend, dict(block_table=_i(2, 5)), I), (extend, dict(seq_lens=_i(2)), I), (extend, dict(softmax_scale=math.inf), I),
    (extend, dict(out=_buffer[:5, :16], q=_buffer[:5, 8:24]), I), (extend, dict(out=_buffer[1:6, :16], q=_buffer[:5, :16]), I),
    (extend, dict(out=torch.as_strided(_buffer, (5, 16, 128), (2048, 64, 1))), I), (extend, dict(device_error=torch.zeros(1)), I),
    (extend, dict(lse=torch.as_strided(_buffer.view(torch.float32), (5, 16), (16, 1)), q=_buffer[:5, :16]), I),
    (write, dict(k_cache=_c(3, 1, 64, 72), v_cache=_c(3, 1, 64, 72)), I), (write, dict(k_cache=_bf(3, 2, 64, 128), v_cache=_bf(3, 2, 64, 128)), I),
    (write, dict(k_cache=_c(3, 2, 64, 128), v_cache=_c(3, 2, 64, 128)), U), (write, dict(k_scale=0.0), I), (write, dict(v_scale=2.0 ** 101), I),
    (write, dict(k_scale=2.0 ** -101), I), (write, dict(v_scale=math.nan), I), (write, dict(q_in=_bf(2, 16, 64)), U),
    (write, dict(slots=_i(3)), I), (write, dict(positions=_i(2).long()), I), (write, dict(rope=None), I), (write, dict(rope=hpc.HpcRope()), I),
    (write, dict(eps=-1.0), I), (write, dict(q_norm_weight=_bf(64)), I), (write, dict(q_out=_buffer[:2, :16], q_in=_buffer[:2, 8:24]), I),
    (write, dict(k_cache=_kv[:, 0], v_cache=_kv[:, 0]), I), (write, dict(k_cache=_kv[:, 0].expand(3, 2, 64, 72)[:1].expand(3, 2, 64, 72), v_cache=_c(1, 2, 64, 72).expand(3, 2, 64, 72)), I),
    (write, dict(device_error=torch.zeros(1)), I), (write, dict(q_out=None), I),
]


def outcome(call, kw):
    try:
        call(**kw)
    except Exception as e:  # noqa: BLE001 (what it is, is compared)
        return type(e), str(e), getattr(e, "status", None)
    return None


@pytest.mark.parametrize("n", range(len(BAD)))
def test_refused_alike_by_both_paths(n, monkeypatch):
    call, kw, status = BAD[n]
    got = outcome(call, kw)
    assert got is not None and got[2] == status, got
    if hpc._native is not None:
        monkeypatch.setattr(hpc, "_native", None)
        assert outcome(call, kw) == got


def test_valid_arguments_reach_the_device():
    """What is not refused asks for a device last of all (there may be none here)."""
    if torch.cuda.is_available():
        pytest.skip("the CPU's tensors are refused where there is a device")
    q, kv = _buffer[:2], _kv
    for call, kw in ((extend, dict()), (extend, dict(lse=None)), (write, dict()),
                     (write, dict(q_in=q[:, :16], k_in=q[:, 16:18], v_in=q[:, 18:20], q_out=q[:, :16], k_cache=kv[:, 0], v_cache=kv[:, 1])),
                     (extend, dict(k_cache=_c(2, 4, 64, 72).transpose(0, 1), v_cache=_c(2, 4, 64, 72).transpose(0, 1)))):
        assert outcome(call, kw)[2] == hpc.HPC_ERR_CUDA
    assert outcome(extend, dict(q=_bf(0, 16, 128), out=_bf(0, 16, 128), lse=None)) is None
    assert outcome(decode, dict(q=_bf(0, 16, 128), out=_bf(0, 16, 128), lse=None, seq_lens=_i(0), block_table=_i(0, 3))) is None


@pytest.mark.parametrize("args,status", [
    ((0, 1, 152, 64), I), ((4, 1, 0, 64), I), ((4, 1, 152, 0), I), ((4, 1, 152, 12), I), ((4, 0, 152, 64), U), ((4, 9, 152, 64), U),
    ((4097, 1, 152, 64), U), ((4, 1, 152, 520), U), ((4, 1, 65536, 64), U)])
def test_plan_creation(args, status):
    with pytest.raises(hpc.HpcError) as e:
        hpc.hpc_decode_kv4_plan_create(*args)
    assert e.value.status == status


@pytest.mark.parametrize("cache", [_c(4, 2, 64, 72), _c(4, 2, 64, 72).view(torch.float8_e4m3fn)])
def test_other_calls_refuse_the_rows(cache):
    """72-byte rows are no e4m3 cache of theirs."""
    for call in (lambda: hpc.hpc_rope_kv_write(_bf(2, 16, 128), _bf(2, 2, 128), _bf(2, 2, 128), _i(2), _i(2), hpc.hpc_rope_init(), _bf(2, 16, 128),
                                               cache, cache.clone(), stream=0),
                 lambda: hpc.hpc_extend_attn(_bf(5, 16, 128), cache, cache, _i(3, 5), _i(3), _i(4), _bf(5, 16, 128), stream=0)):
        with pytest.raises(hpc.HpcError) as e:
            call()
        assert e.value.status in (I, U)


@pytest.mark.parametrize("kw,message", [
    (dict(lse=torch.zeros(5, 1).expand(5, 16)), "lse overlap"), (dict(lse=torch.zeros(1, 16).expand(5, 16)), "lse overlap"),
    (dict(lse=torch.zeros(200).as_strided((5, 16), (15, 1))), "lse overlap"), (dict(out=_bf(1, 16, 128).expand(5, 16, 128)), "out overlap")])
def test_overlapping_results_are_refused(kw, message):
    got = outcome(extend, kw)
    assert got[2] == I and message in got[1]


def test_results_in_other_orders_are_not_refused():
    if torch.cuda.is_available():
        pytest.skip("the CPU's tensors are refused where there is a device")
    for kw in (dict(lse=torch.zeros(16, 5).T), dict(out=_bf(16, 5, 128).transpose(0, 1)), dict(lse=torch.zeros(5, 40)[:, 3:19])):
        assert outcome(extend, kw)[2] == hpc.HPC_ERR_CUDA
