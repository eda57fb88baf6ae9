"""Where moved entries go and which nodes are read for them, at the ends of the ranges (csrc/pace_move_range.h), on the CPU
under AddressSanitizer and UndefinedBehaviorSanitizer: tests/native/test_move_range.cpp."""
import os
import tempfile

from test_native_sanitized import HERE, _build_and_run


def test_moved_ranges_read_nodes_of_their_own_row_only():
    with tempfile.TemporaryDirectory() as d:
        _build_and_run([os.path.join(HERE, "native", "test_move_range.cpp")], d)
