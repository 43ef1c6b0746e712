"""Host-side refusals of the paged cache's C entry points beside those of test_oracle_paged.py (no GPU call)."""
import pytest

from test_oracle_paged import _attn, _cache, _lib

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("scale,cap,word", [
    (0.0, 1e-39, "cap"), (0.0, 1e-19, "cap"), (0.0, 3e38, "cap"), (0.0, 1e19, "cap"), (0.0, INF, "cap"), (0.0, NAN, "cap"),
    (0.0, -1e-30, "cap"), (3e38, 0.0, "scale"), (INF, 0.0, "scale"), (-INF, 0.0, "scale"), (NAN, 0.0, "scale")])
def test_caps_and_scales_whose_quotients_leave_fp32_are_refused(scale, cap, word):
    vx, L = _lib()
    assert _attn(vx, L, _cache(L), opts=(scale, cap, 0, None, None), nws=16) == 1
    assert word in vx.lib.vx_last_error().decode()


@pytest.mark.parametrize("scale,cap", [(0.0, 0.0), (-1.0, 1e18), (1e18, 1e-18), (1e-30, 30.0)])
def test_caps_and_scales_within_the_limits_pass(scale, cap):
    vx, L = _lib()
    assert _attn(vx, L, _cache(L), opts=(scale, cap, 0, None, None), nws=16) == 1      # refused for the workspace alone
    assert "too small" in vx.lib.vx_last_error().decode()
