"""Values that hpc_rope_init's doubles hold and the table's fp32 or the scaled base does not; no GPU is needed."""
import numpy as np
import pytest

import paged_gqa_decode_hpc_gb300 as hpc


@pytest.fixture(scope="module", autouse=True)
def _lib():
    hpc.build()
    hpc.load_library()


@pytest.mark.parametrize("kw", [dict(magnitude=1e39), dict(magnitude=1e-46), dict(scaling="base", factor=1e200, rot_dim=4),
                                dict(scaling="base", base=1e200, factor=1e150)])
def test_refused(kw):
    with pytest.raises(hpc.HpcError) as e:
        hpc.hpc_rope_init(**kw)
    assert e.value.status == hpc.HPC_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,magnitude", [(dict(magnitude=3e38), 3e38), (dict(magnitude=1e-44), 1e-44),
                                          (dict(scaling="base", base=1e100, factor=1e100), 1.0),
                                          (dict(scaling="ramp", factor=1e300, original_len=4096, low=1.0, high=32.0), 0.1 * np.log(1e300) + 1)])
def test_taken(kw, magnitude):
    assert hpc.hpc_rope_init(**kw).magnitude == np.float32(magnitude)
