"""The attention-layer operators' host code (csrc/pace_cache.cpp) under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU, linked against recording stand-ins of the launchers."""
import os
import tempfile

from test_native_sanitized import CSRC, HERE, _build_and_run


def test_cache_entry_points_under_sanitizers():
    with tempfile.TemporaryDirectory() as d:
        _build_and_run([os.path.join(HERE, "native", "test_cache_host_sanitized.cpp"),
                        os.path.join(CSRC, "pace_cache.cpp")], d)
