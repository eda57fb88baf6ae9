"""CPU tests of what the Python binding of the drafts' operators refuses by itself, before any tensor is looked at."""
import inspect

import pytest


@pytest.mark.parametrize("name", ["draft_verify", "prepare_draft_verify"])
def test_verification_names_the_workspace_that_it_needs(name):
    import bit_recurrent_state_amd as pace
    cfg = pace.VerifyConfig(B=1, T=1, V=2)
    assert pace.draft_verify_workspace_bytes(cfg) > 0            # (every call needs some)
    with pytest.raises(ValueError, match="workspace is required"):
        getattr(pace, name)(cfg, *[None] * 7)
    # its place among the arguments
    assert list(inspect.signature(getattr(pace, name)).parameters)[8:] == ["draft", "draft_lens", "workspace", "stream"]
