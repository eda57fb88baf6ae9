"""Commits into buffers whose counts lie outside a period (include/pace.h: read as clamped to it)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_draft import LAYERS, by_steps, layer, make_tokens, run_commit, same_layer  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["pace4", "pace48_mixed", "tiny_f32", "sym8_dP16", "d64_g64_dP1", "bf16_state"])
def test_commits_at_counts_outside_the_period(name):
    dP, B, T = LAYERS[name][8], 8, 11
    held = [dP, dP + 32, 2 ** 31 - 1, -3, -2 ** 31, dP, dP + 1, dP - 1]
    ocfg, gcfg, state, buf = layer(name, 51, B=B, counts=held)
    toks = make_tokens(52, B, T, ocfg.Hv, ocfg.Hk, ocfg.dk, ocfg.dv, bf16=ocfg.bf16_io)
    nodes = np.tile(np.arange(T, dtype=np.int32), (B, 1))
    # nothing is taken: nothing changes
    none = np.array([0, 0, -1, 0, -2 ** 31, -7, 0, 0], dtype=np.int32)
    st, bu = run_commit(gcfg, state, buf, toks, nodes, none)
    assert np.array_equal(st.cpu().numpy(), state) and np.array_equal(bu.cpu().numpy(), buf)
    # some sequences take tokens, others none
    for counts in ([0, 1, 0, 1, 0, 9, 3, 1], [1, 0, 11, 0, 5, 0, 0, 0]):
        counts = np.array(counts, dtype=np.int32)
        got, want = run_commit(gcfg, state, buf, toks, nodes, counts), by_steps(gcfg, state, buf, toks, nodes, counts)
        same_layer(ocfg, got, want)
