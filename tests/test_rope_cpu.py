"""Rotary tables and the refusals of hpc_rope_kv_write, without a GPU."""
import math

import numpy as np
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from oracle import rope_ref as R

I, U = hpc.HPC_ERR_INVALID_ARG, hpc.HPC_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    hpc.build()
    hpc.load_library()


CASES = [dict(scaling="none"), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
         dict(scaling="banded", factor=8.0, original_len=8192, low=1.0, high=4.0),
         dict(scaling="ramp", factor=16.0, original_len=4096, low=1.0, high=32.0)]


@pytest.mark.parametrize("rot_dim", [4, 20, 64, 90, 128])
@pytest.mark.parametrize("base", [1e4, 5e5])
@pytest.mark.parametrize("case", CASES, ids=lambda c: c["scaling"])
def test_tables_match_the_formulas(rot_dim, base, case):
    f, mag = R.frequencies(rot_dim, base, **case)
    t = hpc.hpc_rope_init(rot_dim, True, base, **case)
    got = np.array(t.freq_hi, np.float64) + np.array(t.freq_lo, np.float64)
    # two floats hold 2^-48 of the double, the doubles' own roundings are far below
    assert np.all(np.abs(got[:rot_dim // 2] - f) <= 2.0 ** -47 * f)
    assert np.all(got[rot_dim // 2:] == 0)
    assert abs(t.magnitude - mag) <= 2.0 ** -24 * mag and t.rot_dim == rot_dim and t.interleaved == 1


def test_scalings_at_their_ends():
    none, _ = R.frequencies(128, 1e4)
    for case in CASES[3:]:
        f, _ = R.frequencies(128, 1e4, **case)
        assert f[0] == none[0]                                        # fast pairs stay
        assert abs(f[-1] - none[-1] / case["factor"]) <= 1e-15 * none[-1]  # slow ones are stretched
        assert np.all(np.diff(f) < 0)
    assert hpc.hpc_rope_init(64, False, 1e4, "ramp", 8.0, 4096, 1.0, 32.0, magnitude=1.5).magnitude == 1.5


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=130), dict(rot_dim=63), dict(base=1.0), dict(base=math.inf),
    dict(base=math.nan), dict(scaling="cubic"), dict(scaling="linear", factor=0.5),
    dict(scaling="linear", factor=math.nan), dict(scaling="base", factor=2.0, rot_dim=2),
    dict(scaling="banded", factor=2.0, original_len=0, low=1.0, high=4.0),
    dict(scaling="banded", factor=2.0, original_len=100, low=4.0, high=4.0),
    dict(scaling="ramp", factor=2.0, original_len=100, low=0.0, high=4.0),
    dict(magnitude=-1.0), dict(magnitude=math.inf)])
def test_table_refusals(kw):
    with pytest.raises(hpc.HpcError) as e:
        hpc.hpc_rope_init(**kw)
    assert e.value.status == I


def _args(n=3, hq=8, hkv=2, dtype=torch.bfloat16):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    cache = torch.zeros(4, hkv, 64, 128, dtype=dtype)
    return dict(q_in=z(n, hq, 128), k_in=z(n, hkv, 128), v_in=z(n, hkv, 128),
                positions=torch.zeros(n, dtype=torch.int32), slots=torch.zeros(n, dtype=torch.int32),
                rope=hpc.hpc_rope_init(), q_out=z(n, hq, 128), k_cache=cache, v_cache=cache.clone())


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _off(t, n):
    """t's shape at an address n elements into its buffer."""
    return torch.zeros(t.numel() + n, dtype=t.dtype)[n:].view(t.shape)


@pytest.mark.parametrize("change,status", [
    (dict(q_in=None), I), (dict(q_in=torch.zeros(3, 8, 128)), I), (dict(k_in=_bf(2, 2, 128)), I),
    (dict(v_in=_bf(3, 1, 128)), I), (dict(q_out=_bf(3, 4, 128)), I), (dict(q_in=_bf(3, 7, 128)), I),
    (dict(q_in=_bf(3, 8, 64)), U), (dict(positions=torch.zeros(2, dtype=torch.int32)), I),
    (dict(slots=torch.zeros(3)), I), (dict(slots=None), I),
    (dict(k_cache=_bf(4, 2, 32, 128), v_cache=_bf(4, 2, 32, 128)), U),
    (dict(k_cache=_bf(4, 1, 64, 128), v_cache=_bf(4, 1, 64, 128)), I),
    (dict(v_cache=_bf(5, 2, 64, 128)), I), (dict(k_cache=torch.zeros(4, 2, 64, 128)), I),
    (dict(q_norm_weight=_bf(64)), I), (dict(k_norm_weight=_off(_bf(128), 1)), I),
    (dict(k_norm_weight=torch.zeros(128, dtype=torch.int32)), I),
    (dict(eps=-1.0), I), (dict(eps=math.nan), I),
    (dict(q_in=_off(_bf(3, 8, 128), 4)), I), (dict(q_in=_bf(3, 8, 132)[..., :128]), I),
    (dict(q_in=_bf(3, 128, 8).transpose(1, 2)), I),
    (dict(q_out_fp8=torch.zeros(3, 8, 64, dtype=torch.uint8)), I),
    (dict(q_out_fp8=torch.zeros(3, 8, 128, dtype=torch.uint8), q_fp8_scale=0.0), I),
    (dict(q_out_fp8=_bf(3, 8, 128)), I)])
def test_call_refusals(change, status):
    with pytest.raises(hpc.HpcError) as e:
        hpc.hpc_rope_kv_write(**{**_args(), **change}, stream=0)
    assert e.value.status == status


def test_cache_scale_table_and_alias_refusals():
    a = _args(dtype=torch.uint8)
    bad = [dict(k_scale=0.0), dict(v_scale=math.inf), dict(rope=hpc.HpcRope())]
    t = hpc.hpc_rope_init()
    t.freq_hi[3] = math.nan
    bad.append(dict(rope=t))
    q = _bf(3, 16, 128)
    bad.append(dict(q_in=q[:, :8], q_out=q[:, ::2]))  # q_out starts on q_in with other strides
    for change in bad:
        with pytest.raises(hpc.HpcError) as e:
            hpc.hpc_rope_kv_write(**{**a, **change}, stream=0)
        assert e.value.status == I


def test_no_tokens_is_no_work():
    hpc.hpc_rope_kv_write(**_args(n=0), stream=0)
