"""The ends of the 4-bit attention's ranges: as many query heads as a plan serves, and plans of more CTAs than the merge of
several new tokens looks over at once (512). Tolerances from kv4_util.attend."""
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.kv4_util import Paged, cu_of, decode
from tests.test_gpu_kv4_extend import extend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


@pytest.mark.parametrize("q_len", [1, 2, 7])
@pytest.mark.parametrize("sms", [513, 700, 1100])
def test_more_ctas_than_the_merge_looks_over_at_once(sms, q_len):
    """Enough units that every CTA has a part: pairs are split, and begin, everywhere among the owners."""
    lens = [60000, 9, 41000, 800, 0, 29000, 64]
    c = Paged(lens, hkv=2, q_rows=len(lens) * q_len, seed=sms + q_len)
    c.check(*decode(c, q_len, sms=sms), cu_of([q_len] * len(lens)))


@pytest.mark.parametrize("q_len", [1, 2, 8])
def test_64_kv_heads(q_len):
    c = Paged([300, 0, 70, 1500], hkv=64, q_rows=4 * q_len, seed=q_len)
    c.check(*decode(c, q_len), cu_of([q_len] * 4))


def test_64_kv_heads_of_a_prompt():
    new = [40, 3]
    c = Paged([40, 200], hkv=64, q_rows=43, seed=9)
    c.check(*extend(c, new), cu_of(new))
