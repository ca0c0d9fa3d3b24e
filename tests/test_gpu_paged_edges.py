"""The paged cache operators at the ends of what their arguments may be, against the 64-bit
definitions in paged_ref; bounds as derived in test_gpu_paged."""
import pytest
import torch

from hybrid_attention_ssm_b200 import hymba as H
from tests import paged_ref as R
from tests.test_gpu_paged import check_attention, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.lib()


@pytest.mark.parametrize("M", [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 65])
@pytest.mark.parametrize("W", [5, 2 ** 31 - 1])
def test_meta_count_up_to_the_largest_int(M, W):
    """More meta tokens than any sequence has: every position is visible, whatever the window."""
    lens, ps, Hq, Hkv, D, dt = [0, 1, 5, 6, 64, 257, 3000], 32, 10, 2, 64, torch.float16
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=90)
    q = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(91)).to(dt)
    ref = R.attention(k, v, table, lens, q, D ** -0.5)
    got, lse, status = run_attention(k, v, table, lens, q, n_meta=M, window=W)
    assert status == H.OK
    check_attention(got, lse, ref, v, max(lens), dt, torch.float32, D)
