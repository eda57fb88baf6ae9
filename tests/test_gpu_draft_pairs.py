"""Outputs of drafts and commits in every layout of a layer: kind of state, width, group, buffer, type of the inputs and tiles of
tokens, each of which is a kernel of its own."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_draft as t  # noqa: E402

pytestmark = pytest.mark.gpu


def _layouts():
    for kind, d, group, hb in (("sym", 64, 32, None), ("sym", 64, 64, None), ("sym", 128, 32, None), ("sym", 128, 64, None),
                               ("sym", 64, 64, [4, 8]), ("sym", 128, 64, [8, 4]), ("asym", 64, 32, [8, 4]), ("asym", 128, 32, None),
                               ("asym", 128, 64, [4, 8]), ("bf16", 64, 32, None), ("bf16", 128, 32, None)):
        for buf in ("int8", "mixed") if kind != "bf16" else ("int8",):
            for bf16 in (True, False):
                yield (2, 2, 1, d, group, kind, buf, bf16, 9, hb)


NAMES = {"-".join(str(x) for x in (*y[3:8], "4" if y[9] is None else y[9][0] * 10 + y[9][1])): y for y in _layouts()}


# T: one to six tiles of 16 with the eight buffered tokens that there may be
@pytest.mark.parametrize("T", [3, 8, 24, 40, 56, 64])
@pytest.mark.parametrize("name", list(NAMES))
def test_outputs_in_every_layout(monkeypatch, name, T):
    monkeypatch.setitem(t.LAYERS, name, NAMES[name])
    ocfg, gcfg, state, buf = t.layer(name, 81 + T, counts=[8, 5])
    toks = t.make_tokens(82 + T, ocfg.B, T, ocfg.Hv, ocfg.Hk, ocfg.dk, ocfg.dv, bf16=ocfg.bf16_io)
    par = t.trees(np.random.default_rng(T), ocfg.B, T, "tree")
    lens = [T, (T + 1) // 2]
    o = t.step(gcfg, state, buf, toks, T, t.bits(par), lens)
    t.check_step(ocfg, o, state, buf, toks, t.paths(par), lens, [(0, 0), (1, 1)])


@pytest.mark.parametrize("name", [n for n in NAMES if NAMES[n][5] == "bf16"])
def test_commits_to_states_of_bf16(monkeypatch, name):
    monkeypatch.setitem(t.LAYERS, name, NAMES[name])
    B, T = 4, 21
    ocfg, gcfg, state, buf = t.layer(name, 91, B=B, counts=[0, 3, 8, 7])
    toks = t.make_tokens(92, B, T, ocfg.Hv, ocfg.Hk, ocfg.dk, ocfg.dv, bf16=ocfg.bf16_io)
    nodes = np.tile(np.arange(T, dtype=np.int32), (B, 1))
    counts = np.array([T, 6, 1, 0], dtype=np.int32)
    t.same_layer(ocfg, t.run_commit(gcfg, state, buf, toks, nodes, counts), t.by_steps(gcfg, state, buf, toks, nodes, counts))
