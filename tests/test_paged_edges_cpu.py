"""More refusals of the paged calls, decided on the host (the made-up addresses of
test_paged_cpu are never touched)."""
import pytest

from hybrid_attention_ssm_b200 import build as hbuild
from hybrid_attention_ssm_b200 import hymba as H
from tests.test_paged_cpu import A, append


@pytest.fixture(scope="module", autouse=True)
def _lib():
    hbuild.build()
    H.lib()


def test_queries_in_place_need_the_rows_of_the_output():
    """q_out may be q itself only where a row of one is a row of the other: wider source elements
    or a larger row stride would let one token's result overwrite another's query."""
    for kw in (dict(src=H.DT_F32), dict(src=H.DT_BF16), dict(src=H.DT_F16, qs=264), dict(src=H.DT_F16, qs=512, cu=None)):
        assert append(**{**dict(q=A, q_out=A), **kw}) == H.ERR_INVALID_ARG, kw
