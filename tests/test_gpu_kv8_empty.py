"""Selection without query rows: the lists of blocks that no sequence has are filled with -1."""
import pytest
import torch

import test_gpu_kv8 as base
from test_gpu_kv8 import Both, cumulative, ints

pytestmark = pytest.mark.gpu
_need_gpu = base._need_gpu


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("other_stream", [False, True])
def test_select_without_rows_fills_the_lists(given, other_stream):
    x = Both(3, 4, 2, 64, 32, "int8", seed=50)
    x.fill_up([100, 60, 1])
    q = x.rows(0, 4)
    lists = torch.full((3, 5, 2, 6), 77, dtype=torch.int32, device=base.DEV) if given else None
    torch.full((3, 5, 2, 6), 78, dtype=torch.int32, device=base.DEV)  # (memory that is used again)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if other_stream else None
    got = x.cache.select(q, ints(x.table), ints(x.held), cumulative([0, 0, 0]), 20, 128, 4, 6, 1, 1,
                         blocks=lists, stream=stream)
    torch.cuda.synchronize()
    assert got.shape == (3, 5, 2, 6) and (got == -1).all()
    if given:
        assert got.data_ptr() == lists.data_ptr()
    out, lse = x.cache.attend(q, ints(x.table), ints(x.held), cumulative([0, 0, 0]), 20, 128,
                              blocks=got, q_block=4)
    assert out.shape == q.shape and lse.shape == (0, 4)


def test_select_without_rows_on_a_raw_stream_and_in_a_graph():
    x = Both(1, 4, 1, 64, 32, "int8", seed=51)
    x.fill_up([100])
    q, stream = x.rows(0, 1), torch.cuda.Stream()
    args = (ints(x.table), ints(x.held), cumulative([0]), 8, 128, 8, 3)
    lists = torch.full((1, 1, 1, 3), 77, dtype=torch.int32, device=base.DEV)
    work = torch.empty(0, dtype=torch.uint8, device=base.DEV)
    torch.cuda.synchronize()
    x.cache.select(q, *args, blocks=lists, workspace=work, stream=stream.cuda_stream)
    torch.cuda.synchronize()
    assert (lists == -1).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = x.cache.select(q, *args)
    for fill in (5, 6, 7):
        got.fill_(fill)
        graph.replay()
        torch.cuda.synchronize()
        assert (got == -1).all()


def test_select_without_rows_is_checked_like_others():
    from diffusion_activation_residual_amd import cfz
    x = Both(1, 4, 1, 64, 32, "int8", seed=52)
    args = (x.rows(0, 1), ints(x.table), ints([0]), cumulative([0]), 8)
    for kw in (dict(max_kv=129, q_block=8, count=3), dict(max_kv=128, q_block=8, count=3, first=2, last=2)):
        with pytest.raises(cfz.CfzError):
            x.cache.select(*args, **kw)
