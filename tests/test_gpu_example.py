"""The hybrid-stack example: gated-delta layers and an attention layer with its rotary positions and
quantised cache, through prompt, decode and a tree of drafts.  Its forms agree up to the order
of fp32 sums (other waves, pieces and kernels: under 2^-16 of the largest value) and bf16
rounding of outputs that then differ by a step (2^-7) at most where a sum lies next to a tie; the
residual and the projection that follow round to bf16 once more each, half a step of 2^-8."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_hybrid_example_forms_agree():
    import hybrid_decode
    found = hybrid_decode.main()
    assert len(found) == 3
    for name, value in found.items():
        assert value <= 2.0 ** -7 + 2 * 2.0 ** -8 + 2.0 ** -16, (name, value)
