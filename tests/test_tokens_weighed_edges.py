"""Weighed attention at the edges of its contract: plans of a given split."""
import pytest

from conv_bn_silu_gb300 import _binding as B
from tests.test_tokens_refusals import desc


@pytest.fixture(scope="module", autouse=True)
def token_calls(cuda_lib):
    from conv_bn_silu_gb300 import build
    build.build_tokens()


def test_a_given_split_stays(cuda_lib):
    """force_split of the few-row kernel is its number of ranges, over eight too."""
    for kw in (dict(heads=8), dict(heads=8, cache_prec=B.CBS_BF16, force_kernel=B.CBS_ATTN_ROWS)):
        plan = B.cbs_weighed_plan(desc(batch=1, max_len=8000, force_split=20, **kw))
        assert (plan.attention.kernel, plan.attention.split) == (B.CBS_ATTN_ROWS, 20), kw
    plan = B.cbs_weighed_plan(desc(batch=1, max_len=8000, heads=8))
    assert (plan.attention.kernel, plan.attention.split) == (B.CBS_ATTN_CLUSTER, 8)
