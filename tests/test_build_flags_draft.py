"""How the sources of the drafts' operators are compiled (bit_recurrent_state_amd/build.py)."""
import os

from test_build_flags import PACKAGE, _build


def test_verification_and_moves_honour_nan():
    """pace_draft.h says what verification makes of probabilities and uniforms that are NaN; moves may move anything."""
    b = _build()
    for src in b.SOURCES:
        text = open(os.path.join(PACKAGE, "csrc", src)).read()
        if "pace_draft_verify(" in text or "launch_draft_verify(" in text or "launch_cache_move(" in text:
            assert src in b.HONOR_NANS, src
    assert {"pace_draft.cpp", "pace_draft_verify.hip", "pace_cache_move.hip"} <= b.HONOR_NANS
