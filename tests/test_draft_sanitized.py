"""The host code of the operators that serve drafted tokens (csrc/pace_draft.cpp) under AddressSanitizer
and UndefinedBehaviorSanitizer, over random and extreme sizes, linked against recording stand-ins of the
kernel launchers: tests/native/test_draft_host_sanitized.cpp."""
import os
import tempfile

from test_native_sanitized import CSRC, HERE, _build_and_run


def test_draft_entry_points_under_sanitizers():
    with tempfile.TemporaryDirectory() as d:
        _build_and_run([os.path.join(HERE, "native", "test_draft_host_sanitized.cpp"),
                        *(os.path.join(CSRC, n) for n in ("pace_draft.cpp", "pace_host.cpp", "pace_cache.cpp"))], d)
