"""GPU tests of the 8-bit K/V cache where a row that must not count holds what
would spoil the others: zero rows moved between blocks whose scales lie far
apart."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import fp4_kv_cache_rope_gb300 as K  # noqa: E402
from oracle import kv8 as O  # noqa: E402
from kv8_tools import Pair  # noqa: E402


@pytest.mark.parametrize("into", ["place", "cache"])
@pytest.mark.parametrize("fmt", [O.E4M3, O.INT8])
@pytest.mark.parametrize("block,page,D", [(16, 16, 64), (64, 0, 128), (128, 128, 64)])
def test_evict_keeps_zero_rows_zero_beside_rows_far_smaller(block, page, D, fmt, into):
    """Zero rows come out of a block with a large scale into one whose other rows
    are 2^-20 to 2^-200 as large."""
    for big, small in ((2.0 ** 5, 2.0 ** -15), (2.0 ** 9, 2.0 ** -22), (2.0 ** 9, 2.0 ** -24),
                       (2.0 ** 20, 2.0 ** -25), (2.0 ** 100, 2.0 ** -100)):
        n, keep = 2 * block, block
        p = Pair(1, 2, D, n, block, page, fmt, seed=91)
        ws = p.c.workspace(1, 2)
        k, v = (p.rows(n, 2, "f32") for _ in "kv")
        for x, at in ((k, 0), (v, 1)):
            x[:, :block] = 0
            x[:, at] = big                      # the one row of the first block that is not 0
            x[:, block:] *= small
        p.append(k, v, ws)
        w = np.ones(n)
        w[: 2] = 0.0                            # it goes, zero rows and small ones stay
        w[2 + block // 2: block] = 0.0
        w[n - 2:] = 0.0
        p.set_mass([[w] * 2])
        kept = torch.empty(1, 2, keep, dtype=torch.int32, device="cuda")
        rows = O.evict(w, n, keep, 0, 0)
        d = p
        if into == "cache":
            d = Pair(1, 2, D, keep, block, page, fmt, seed=92)
        K.kv8_evict(p.c, keep, 0, 0, kept, ws, dst=None if d is p else d.c)
        for h in range(2):
            assert kept[0, h].tolist() == rows.tolist()
            for s in "kv":
                d.seq[0, h, s] = p.seq[0, h, s].keep(rows)
        d.len = [keep]
        d.check()
        assert K.get_status(ws) == 0
