"""The scales that kda_attn_fwd takes and refuses, on the CPU."""
from __future__ import annotations

import pytest

import gated_delta_rule_62_amd as kda
from tests.test_serving_boundary import ATTN, ATTN_BASE, _call, lib  # noqa: F401  (a fixture)


@pytest.mark.parametrize("scale,status", [
    (0.0, kda.KDA_OK), (-0.0, kda.KDA_OK), (1e-45, kda.KDA_OK), (2.35e38, kda.KDA_OK),
    # scale log2(e) beyond the largest float: scores of zero times it would be NaN
    (2.37e38, kda.KDA_ERR_BAD_SCALE), (3.4e38, kda.KDA_ERR_BAD_SCALE),
    (-1e-45, kda.KDA_ERR_BAD_SCALE)])
def test_scale_limits(lib, scale, status):  # noqa: F811
    assert _call(lib.kda_attn_fwd_check, ATTN, ATTN_BASE, scale=scale) == status
