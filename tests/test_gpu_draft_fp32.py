"""Precision of the outputs of drafts in fp32: a state's codes go into the sums as the values that they stand for, so that
what a code's offset would be has no roundings there."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import packing as pk  # noqa: E402
from pace_synth import random_packed_state_parts  # noqa: E402
from test_gpu_draft import bits, layer, make_tokens, step, trees  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 6, 20, 50])
@pytest.mark.parametrize("which", ["all", "some"])
@pytest.mark.parametrize("name", ["pace48_int8_f32", "tiny_f32", "f32_g32_mixed_dP32"])
def test_codes_at_their_zero_points_have_no_part_whatever_their_scales(name, which, T):
    """All groups, or every other one: the outputs are, bit for bit, those of the same state with scales of zero there."""
    ocfg, gcfg, _, buf = layer(name, 61)
    parts = random_packed_state_parts(62, ocfg.B, ocfg.Hv, ocfg.dk, ocfg.dv, ocfg.group, [ocfg.bits(h) for h in range(ocfg.Hv)],
                                      ocfg.asym)
    bare = []
    for row in parts:
        bare.append([])
        for h, (codes, scales, zeros) in enumerate(row):
            G = slice(None, None, 1 if which == "all" else 2)
            none = scales.copy()
            none[G], scales[G] = 0.0, 2.0 ** 14 * scales[G]
            z = np.repeat(zeros, ocfg.group, axis=0) if ocfg.asym else np.full_like(codes, 1 << (ocfg.bits(h) - 1))
            there = np.zeros(len(scales), dtype=bool)
            there[G] = True
            codes[np.repeat(there, ocfg.group)] = z[np.repeat(there, ocfg.group)]
            bare[-1].append((codes, none, zeros))
    states = [pk.pack_state(ocfg, pk.state_from_parts(ocfg, x)) for x in (parts, bare)]
    assert not np.array_equal(*states)
    toks = make_tokens(63, ocfg.B, T, ocfg.Hv, ocfg.Hk, ocfg.dk, ocfg.dv)
    tree = bits(trees(np.random.default_rng(T), ocfg.B, T, "tree"))
    got, want = (step(gcfg, s, buf, toks, T, tree) for s in states)
    assert torch.equal(got, want) and bool(want.any())
