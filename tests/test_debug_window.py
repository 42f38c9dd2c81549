"""The debug build on the operators over heads and on windowed attention: the release build's bits, no check failing."""
import pytest

from test_debug_build import run

pytestmark = pytest.mark.gpu


def test_debug_and_release_builds_give_the_same_bits():
    from invariant_deterministic_bi_gb300 import _build
    _build.build(debug=True)
    rel, dbg = run("_debug_window_ops.py", debug=False), run("_debug_window_ops.py", debug=True)
    assert rel.pop("debug_build") is False and dbg.pop("debug_build") is True
    assert dbg["status"] == "BI_OK", "a bounds check failed on valid inputs"
    assert dbg == rel
