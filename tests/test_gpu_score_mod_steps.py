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


@pytest.mark.parametrize("modified", [False, True])
@pytest.mark.parametrize("kv,heads", [("q8", (32, 8, 128)), ("q4", (32, 8, 128)), ("q8", (8, 8, 64))])
def test_a_widened_history_does_not_depend_on_what_the_workspace_held(heads, modified, kv):
    """Prompt chunks over a block-scaled pool read a scratch pool through a scratch block table that the kernel before
    fills: the same bits whatever an earlier call left there, called one behind another and replayed."""
    hq, hkv, d = heads
    w = W.random_step(43, [(40, 1500), (90, 600), (33, 2100), (200, 200), (1, 700)], num_q_heads=hq, num_kv_heads=hkv, head_dim=d)
    mod = B.ScoreMod(window=900) if modified else None
    want, ds = _run(w, mod, kv)
    graph = torch.cuda.CUDAGraph()
    fills = (0, 255, 1)
    got = torch.empty((2 * len(fills),) + tuple(ds.out.shape), dtype=ds.out.dtype, device="cuda")

    def calls(at):
        for i, fill in enumerate(fills):
            ds.workspace.fill_(fill)
            R.run_attention(ds)
            got[at + i].copy_(ds.out)

    calls(0)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        calls(len(fills))
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert B.pkv_check_device_status(ds.status) == 0
    assert all(np.array_equal(o.float().cpu().numpy(), want) for o in got)
