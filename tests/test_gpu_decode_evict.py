"""Eviction by accumulated attention weight against an exact entry-by-entry computation (needs a
GB300): whole numbers and moved weights are compared bit for bit."""
import numpy as np
import pytest
import torch

import residual_stream_norm_gb300 as rsn
from tests import _decode_ref as ref
from tests._gpu import lib

pytestmark = pytest.mark.gpu


def guarded(shape, dtype, value):
    n = int(np.prod(shape))
    buf = torch.full((n + 256,), value, dtype=dtype, device="cuda")
    return buf, buf[128:128 + n].view(*shape)


def check(table, lens, weight, budget, recent, freed_extra=0, in_place=False):
    rows, width = table.shape
    F = max(0, width - budget) + freed_extra
    dt, dn, dw = (torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (table, lens, weight))
    bufs = [guarded((rows, width), torch.int64, -77), guarded((rows,), torch.int32, -77),
            guarded((rows, width), torch.float32, -77.0), guarded((rows, F), torch.int64, -77)]
    outs = [b[1] for b in bufs]
    if in_place:
        for o, x in zip(outs, (dt, dn, dw)):
            o.copy_(x)
        dt, dn, dw = outs[:3]
    rsn.beam_kv_evict_fwd(*outs[:3], outs[3] if F else None, dt, dn, dw, budget, recent)
    torch.cuda.synchronize()
    for buf, _ in bufs:
        assert bool((buf[:128] == -77).all()) and bool((buf[-128:] == -77).all()), "guard band"
    want = ref.evict(table, lens, weight, budget, recent, F)
    for name, got, exp in zip(("table", "len", "weight", "freed"), outs, want):
        got = got.cpu().numpy()
        if got.dtype == np.float32:
            got, exp = got.view(np.uint32), exp.view(np.uint32)
        assert np.array_equal(got, exp), f"{name}: {np.argwhere(got != exp)[:5].tolist()}"


def case(rows, width, seed, kind="many"):
    g = np.random.default_rng(seed)
    table = g.integers(0, 2 ** 40, (rows, width))
    if kind == "ties":
        weight = g.integers(0, 4, (rows, width)).astype(np.float32)
    elif kind == "equal":
        weight = np.full((rows, width), 0.25, np.float32)
    else:
        weight = (g.random((rows, width)) ** 8 * 50).astype(np.float32)
    return table, weight


@pytest.mark.parametrize("kind", ["many", "ties", "equal"])
@pytest.mark.parametrize("width,budget,recent", [
    (1, 0, 0), (1, 1, 1), (2, 1, 0), (2, 1, 1), (33, 32, 5), (100, 40, 40), (100, 40, 0),
    (1023, 1000, 7), (1024, 1, 1), (1025, 1024, 100), (2500, 1300, 300), (64, 100, 3)])
def test_sizes(width, budget, recent, kind):
    lib()
    table, weight = case(5, width, width + recent, kind)
    lens = np.array([width, max(0, width - 1), min(budget, width), 0, width + 9], np.int32)
    check(table, lens, weight, budget, recent)
    check(table, lens, weight, budget, recent, freed_extra=3, in_place=True)


def test_negative_length_is_empty():
    lib()
    table, weight = case(2, 50, 1)
    check(table, np.array([-5, 50], np.int32), weight, 20, 4)


def test_signs_nan_and_infinities():
    lib()
    table, weight = case(6, 300, 2)
    weight[0, ::3] = np.nan
    weight[1, :] = np.nan
    weight[2, ::2] = -np.inf
    weight[2, 1::4] = np.inf
    weight[3, :] = 0.0
    weight[3, ::5] = -0.0                  # equal to +0: the lower index stays
    weight[4] = -weight[4]
    weight[5, ::7] = 1e-45
    check(table, np.full(6, 300, np.int32), weight, 120, 10)
    check(table, np.full(6, 300, np.int32), weight, 250, 0)


@pytest.mark.parametrize("kind", ["many", "ties"])
def test_long_rows(kind):
    lib()
    for width, budget, recent, lens in ((40000, 30000, 1000, [40000, 30001]),
                                        (70000, 66000, 0, [70000, 69999]),
                                        (131072, 131000, 64, [131072, 131001])):
        table, weight = case(2, width, width, kind)
        check(table, np.array(lens, np.int32), weight, budget, recent)
        check(table, np.array(lens, np.int32), weight, budget, recent, in_place=True)


def test_many_rows():
    lib()
    table, weight = case(700, 200, 5)
    lens = np.random.default_rng(6).integers(0, 201, 700).astype(np.int32)
    check(table, lens, weight, 100, 20, in_place=True)


def test_no_rows_and_no_width():
    lib()
    e = torch.empty
    for rows, width in ((0, 10), (3, 0)):
        n = torch.full((rows,), 5, dtype=torch.int32, device="cuda")
        t = e((rows, width), dtype=torch.int64, device="cuda")
        w = e((rows, width), device="cuda")
        rsn.beam_kv_evict_fwd(t, n, w, None, t, n, w, 10, 2)
        torch.cuda.synchronize()
        assert bool((n == 0).all())


def test_rows_past_the_shared_memory_of_a_block():
    # more entries a block than it holds weights for, in too many rows for clusters
    lib()
    rows, width, budget, recent = 81, 53000, 52000, 500
    g = np.random.default_rng(7)
    table = g.integers(0, 2 ** 40, (rows, width))
    weight = g.integers(0, 3000, (rows, width)).astype(np.float32)   # many ties
    weight[1] = (g.random(width) ** 8 * 50).astype(np.float32)
    lens = np.full(rows, width, np.int32)
    lens[2], lens[3], lens[4] = budget + 1, budget, 51201
    F = width - budget
    want = [np.full((rows, width), -1, np.int64), np.minimum(lens, budget),
            np.zeros((rows, width), np.float32), np.full((rows, F), -1, np.int64)]
    for r in range(rows):
        n = int(lens[r])
        stay = np.ones(n, bool)
        if n > budget:
            old = n - recent
            order = np.argsort(-weight[r, :old], kind="stable")
            stay[:old] = False
            stay[order[:budget - recent]] = True
        m = int(stay.sum())
        want[0][r, :m], want[2][r, :m] = table[r, :n][stay], weight[r, :n][stay]
        want[3][r, :n - m] = table[r, :n][~stay]
    for in_place in (False, True):
        dt, dn, dw = (torch.from_numpy(x.copy()).cuda() for x in (table, lens, weight))
        outs = [dt, dn, dw] if in_place else [torch.empty_like(x) for x in (dt, dn, dw)]
        outs.append(torch.empty((rows, F), dtype=torch.int64, device="cuda"))
        rsn.beam_kv_evict_fwd(*outs, dt, dn, dw, budget, recent)
        torch.cuda.synchronize()
        for name, got, exp in zip(("table", "len", "weight", "freed"), outs, want):
            assert np.array_equal(got.cpu().numpy(), exp), (name, in_place)


@pytest.mark.parametrize("rows,width", [(15, 100000), (36, 100000), (76, 40000)])
def test_one_more_row_does_not_double_the_time(rows, width):
    # around the numbers of clusters that are resident at once
    lib()

    def time(n):
        table, weight = case(n, width, n)
        dt, dw = torch.from_numpy(table).cuda(), torch.from_numpy(weight).cuda()
        dn = torch.full((n,), width, dtype=torch.int32, device="cuda")
        budget = width - 2000
        outs = [torch.empty_like(x) for x in (dt, dn, dw)]
        outs.append(torch.empty((n, 2000), dtype=torch.int64, device="cuda"))
        graph = torch.cuda.CUDAGraph()
        rsn.beam_kv_evict_fwd(*outs, dt, dn, dw, budget, 100)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            for _ in range(10):
                rsn.beam_kv_evict_fwd(*outs, dt, dn, dw, budget, 100)
        times = []
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    few, more = time(rows), time(rows + 1)
    assert more < 1.75 * few, (few, more)
