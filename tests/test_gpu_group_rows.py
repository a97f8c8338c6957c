"""gemm_group_rows against numpy's stable sort: every value exact."""
import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib

pytestmark = pytest.mark.gpu


def expected(ids, groups):
    kept = (ids >= 0) & (ids < groups)
    key = np.where(kept, ids, np.int64(groups)).astype(np.int64)
    order = np.argsort(key, kind="stable").astype(np.int32)
    n = int(kept.sum())
    order[n:] = -1
    offsets = np.concatenate([[0], np.cumsum(np.bincount(ids[kept], minlength=groups))])
    position = np.full(len(ids), -1, np.int32)
    position[order[:n]] = np.arange(n, dtype=np.int32)
    return offsets.astype(np.int32), order, position


@pytest.mark.parametrize("rows,groups", [
    (0, 3), (1, 1), (1, 5), (31, 7), (32, 64), (33, 1), (1000, 1024), (1025, 8), (8192, 64),
    (8193, 64), (8200, 1500), (9000, 1024), (40000, 2500), (65537, 3), (131072, 128),
    (700001, 257)])
@pytest.mark.parametrize("shape", ["uniform", "skewed", "dropped", "one"])
def test_matches_a_stable_sort(rows, groups, shape):
    rng = np.random.default_rng(rows * 7 + groups)
    if shape == "uniform":
        ids = rng.integers(0, groups, rows)
    elif shape == "skewed":
        ids = np.minimum((groups * rng.random(rows) ** 4).astype(np.int64), groups - 1)
    elif shape == "dropped":
        ids = rng.integers(-2, groups + 3, rows)
        if rows:
            ids[rng.integers(0, rows)] = -2 ** 31
            ids[rng.integers(0, rows)] = 2 ** 31 - 1
    else:
        ids = np.full(rows, groups - 1)
    ids = ids.astype(np.int32)
    got = lib.group_rows(torch.from_numpy(ids).cuda(), groups)
    torch.cuda.synchronize()
    for name, g, e in zip(("offsets", "order", "position"), got, expected(ids, groups)):
        assert np.array_equal(g.cpu().numpy(), e), name


def test_without_positions_and_inside_the_buffers():
    rng = np.random.default_rng(3)
    ids = rng.integers(-1, 9, 5000).astype(np.int32)
    offsets = torch.full((10 + 8,), 77, dtype=torch.int32, device="cuda")
    order = torch.full((5000 + 8,), 77, dtype=torch.int32, device="cuda")
    lib.gemm_group_rows(5000, 9, torch.from_numpy(ids).cuda(), offsets, order)
    e = expected(ids, 9)
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([e[0], [77] * 8]))
    assert np.array_equal(order.cpu().numpy(), np.concatenate([e[1], [77] * 8]))


def test_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(4)
    a, b = (rng.integers(0, 30, 20000).astype(np.int32) for _ in range(2))
    ids = torch.from_numpy(a).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = lib.group_rows(ids, 30)
    side.synchronize()
    for g, e in zip(got, expected(a, 30)):
        assert np.array_equal(g.cpu().numpy(), e)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib.group_rows(ids, 30)
    ids.copy_(torch.from_numpy(b))
    graph.replay()
    torch.cuda.synchronize()
    for g, e in zip(out, expected(b, 30)):
        assert np.array_equal(g.cpu().numpy(), e)
