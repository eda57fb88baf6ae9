"""Attention of many rows in every kind, head width, group and type: several blocks of one and of two
row tiles, as a chain and as trees, ragged.  Scene and tolerances are those of tests/test_gpu_cache.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_cache import STORE, Scene  # noqa: E402

pytestmark = pytest.mark.gpu


def _trees(rng, B, T):
    return [[int(rng.integers(max(-1, i - 5), i)) if i else -1 for i in range(T)] for _ in range(B)]


@pytest.mark.parametrize("kind,d,g", STORE)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,gamma", [(11, 4), (34, 4)])
def test_many_rows_in_every_layout(kind, d, g, bf16, T, gamma):
    """44 rows, past one tile of 32 bf16 rows, and 136, past the 128 fp32 rows of one tile a wave with d = 128."""
    print(f"[cache] rows {kind} d={d} g={g} bf16={bf16} T={T}", flush=True)
    s = Scene(d + g + T, 3, 1, gamma, d, kind, g, 16, [T, 60 + T, 170 + T], bf16)
    s.check(T, [0, 60, 170])
    s.check(T, [0, 60, 170], drafts=[T, 3, T // 2], parents=_trees(np.random.default_rng(T), 3, T))


@pytest.mark.parametrize("kind,d,g", [("fp8", 128, 128), ("int4", 128, 32), ("int8", 256, 64), ("fp8", 64, 32)])
@pytest.mark.parametrize("bf16", [True, False])
def test_many_rows_over_a_cut_context(kind, d, g, bf16):
    """Two row tiles (one with d = 256), pieces over workgroups and absent pages among them."""
    s = Scene(d + g, 1, 1, 4, d, kind, g, 64, [1300], bf16)
    T = 34
    s.check(T, [1300 - T], max_len=1300, rows=[0, 1, 7, 8, 15, 16, 31, 32, 33])
    table = s.table_h.copy()
    table[0, 3], table[0, 20] = -1, s.cfg.num_pages
    s.table = torch.from_numpy(table).cuda()
    hidden = [[p for e in (3, 20) for p in range(64 * e, 64 * e + 64)]]
    s.check(T, [1300 - T], max_len=1300, hidden=hidden, rows=[0, 7, 33])
