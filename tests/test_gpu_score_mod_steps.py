"""Modified scores among their neighbours: other segments of the step, other calls on the stream, other lists."""

import numpy as np
import pytest

import oracle
from continuous_batching_paged_pkv_gb300 import binding as B
from continuous_batching_paged_pkv_gb300 import build as libbuild
from continuous_batching_paged_pkv_gb300 import runtime as R
from continuous_batching_paged_pkv_gb300 import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    libbuild.build()
    oracle.build()


def _slopes(hq):
    return 2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)


def _run(w, mod, kv="bf16"):
    ds = R.prepare(w, kv=kv, mod=mod)
    R.run_step(ds)
    torch.cuda.synchronize()
    assert B.pkv_check_device_status(ds.status) == 0
    return R.out_f32(ds), ds


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("rows", [509, 203, 33])
def test_a_capped_chunk_does_not_depend_on_the_rows_behind_it(rows, biased, d):
    """A chunk whose last warp is partly filled: the same bits alone, before another chunk whose queries lie far beyond
    the cap (their rows are in the chunk's last query tile), and before such decode rows."""
    heads = dict(num_q_heads=32, num_kv_heads=8, head_dim=d)
    mod = B.ScoreMod(softcap=50.0, alibi_slopes=_slopes(32) if biased else None)
    first = W.random_step(31, [(rows, rows + 700)], max_slots=4, **heads)
    want, _ = _run(first, mod)
    for behind in ([(40, 90)], [(1, 700), (1, 64)], [(64, 64), (1, 300), (1, 41)]):
        w = W.random_step(32, [(rows, rows + 700)] + behind, max_slots=4, **heads)
        w.hist_k[0], w.hist_v[0] = first.hist_k[0], first.hist_v[0]
        q = 30.0 * W.bf16_bits_to_f32(w.q)
        q[:rows] = W.bf16_bits_to_f32(first.q)
        w.q = W.f32_to_bf16_bits(q)
        got, _ = _run(w, mod)
        differ = (got[:rows] != want).any((1, 2)).nonzero()[0]
        assert not len(differ), f"behind it {behind}: rows {differ} differ"
