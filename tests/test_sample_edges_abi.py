"""Host-side refusals of headloss_sample at the ends of fp32's range: no GPU, and no address is
dereferenced."""
import pytest

from tests.test_step_ops_abi import ARG, lib, sample  # noqa: F401


@pytest.mark.parametrize("other", [dict(scale=2.37e38), dict(scale=3.4e38), dict(softcap=2.9e-39),
                                   dict(softcap=1e-45)])
def test_sample_refuses_factors_past_fp32(lib, other):  # noqa: F811
    """1 / softcap or logits_scale log2(e) is infinite: such rows have no mass anywhere."""
    assert sample(lib, **other) == ARG


@pytest.mark.parametrize("other", [dict(scale=2.35e38), dict(scale=1e-45), dict(softcap=2.95e-39),
                                   dict(softcap=3.4e38)])
def test_sample_takes_what_fp32_holds(lib, other):  # noqa: F811
    assert sample(lib, N=0, **other) == 0
