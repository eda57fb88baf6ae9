"""The attention-layer operators' host code (csrc/pace_cache.cpp) at the ends of its ranges, under
AddressSanitizer and UndefinedBehaviorSanitizer on the CPU."""
import os
import tempfile

from test_native_sanitized import CSRC, HERE, _build_and_run


def test_cache_limits_under_sanitizers():
    with tempfile.TemporaryDirectory() as d:
        _build_and_run([os.path.join(HERE, "native", "test_cache_limits_sanitized.cpp"),
                        os.path.join(CSRC, "pace_cache.cpp")], d)
