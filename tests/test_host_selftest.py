"""Failure-path self-tests that do not exist are refused before any device work."""
import pytest

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk


@pytest.mark.parametrize("which", [-1, 5, 8, 100])
def test_unknown_selftests(which):
    pbuild.build()
    assert dk.load().dualkv_selftest_kernel(which, 50_000_000, None) == dk.DUALKV_ERR_INVALID
    assert dk.load().dualkv_selftest_kernel(6, 10, None) == dk.DUALKV_ERR_INVALID
