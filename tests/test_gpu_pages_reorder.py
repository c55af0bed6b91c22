"""Reordering of pages in place against a row-by-row model."""
from __future__ import annotations

import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import api  # noqa: E402

DEV = "cuda"


def model(slots, parents, pages):
    """(new slots, copies as (from, to), how many branches found no page)"""
    n = len(slots)
    page = [s if 0 <= s < pages else -1 for s in slots]
    par = [p if 0 <= p < n and page[p] >= 0 else -1 for p in parents]
    free = [page[i] for i in range(n) if page[i] >= 0 and i not in par]
    new, copies, missing, seen = [-1] * n, [], 0, set()
    for i, p in enumerate(par):
        if p < 0:
            continue
        if p not in seen:
            new[i] = page[p]
        elif free:
            new[i] = free.pop(0)
            copies.append((page[p], new[i]))
        else:
            missing += 1
        seen.add(p)
    for i, p in enumerate(par):
        if p < 0 and free:
            new[i] = free.pop(0)
    return new, copies, missing


def run(slots, parents, pools, pages):
    was = [p.clone() for p in pools]
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    got, missing = api.pages_reorder(t(slots), t(parents), pools)
    new, copies, want_missing = model(slots, parents, pages)
    assert got.tolist() == new and int(missing) == want_missing
    for now, old in zip(pools, was):
        for a, b in copies:
            old[b] = old[a]
        assert torch.equal(now, old)


def pools_of(pages, sizes, dtype=torch.float32):
    return [torch.randn(pages, n, device=DEV).to(dtype) for n in sizes]


@pytest.mark.parametrize("rows", [1, 2, 5, 31, 1024, 1025, 3000])
@pytest.mark.parametrize("kind", ["any", "own item", "one", "same", "none"])
def test_rows(rows, kind):
    r = random.Random(rows)
    pages = rows + 7
    slots = r.sample(range(pages), rows)
    parents = {"any": [r.randrange(rows) for _ in range(rows)],
               "own item": [min(rows - 1, i - i % 4 + r.randrange(4)) for i in range(rows)],
               "one": [rows // 2] * rows, "same": list(range(rows)), "none": [-1] * rows}[kind]
    run(slots, parents, pools_of(pages, [24, 8]), pages)


def test_rows_without_pages_and_without_parents():
    r = random.Random(1)
    for rows in (3, 17, 400, 2000):
        pages = rows
        for _ in range(5):
            slots = r.sample(range(pages), rows)
            for i in range(rows):
                if r.random() < 0.3:
                    slots[i] = r.choice([-1, pages, 1 << 30, -5])
            parents = [r.choice([-1, rows, r.randrange(rows), r.randrange(rows)]) for _ in range(rows)]
            run(slots, parents, pools_of(pages, [4]), pages)


@pytest.mark.parametrize("sizes,dtype", [([1], torch.uint8), ([3, 5], torch.bfloat16), ([5000], torch.float32), ([4096] * 24, torch.float32),
                                         ([100003], torch.uint8), ([8] * 128, torch.float16)])
def test_pools(sizes, dtype):
    r = random.Random(3)
    slots = r.sample(range(40), 32)
    pools = [torch.randint(0, 256, (40, n), device=DEV).to(dtype) for n in sizes]
    run(slots, [r.randrange(32) for _ in range(32)], pools, 40)


def test_nothing():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    got, missing = api.pages_reorder(e, e, torch.zeros(3, 4, device=DEV))
    assert got.numel() == 0 and int(missing) == 0
    got, missing = api.pages_reorder(torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV), [])
    assert got.tolist() == [-1, -1] and int(missing) == 0   # no pools, no pages


def test_shapes_out_and_refusals():
    slots = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3)
    parents = torch.tensor([[1, 1, 0], [5, 3, 5]], dtype=torch.int32, device=DEV)
    pool, out = torch.arange(6.0, device=DEV)[:, None].repeat(1, 4), torch.empty_like(slots)
    got, _ = api.pages_reorder(slots, parents, pool, out=out)
    assert got is out and out.tolist() == [[1, 2, 0], [5, 3, 4]]
    assert pool[:, 0].tolist() == [0, 1, 1, 3, 5, 5]
    with pytest.raises(ValueError, match="parent"):
        api.pages_reorder(slots, parents[0], pool)
    with pytest.raises(ValueError, match="shape"):
        api.pages_reorder(slots, parents, pool, out=out.view(3, 2))
    with pytest.raises(Exception, match="failed"):
        api.pages_reorder(slots, parents, pool, out=slots)


def test_captured_on_changing_parents_and_another_stream():
    r = random.Random(5)
    pages, rows = 50, 40
    slots = torch.tensor(r.sample(range(pages), rows), dtype=torch.int32, device=DEV)
    parents = torch.zeros(rows, dtype=torch.int32, device=DEV)
    pools = pools_of(pages, [64, 7])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    api.pages_reorder(slots, torch.arange(rows, dtype=torch.int32, device=DEV), pools, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new, _ = api.pages_reorder(slots, parents, pools)
        slots.copy_(new)
    now, old = slots.tolist(), [p.clone() for p in pools]
    for _ in range(6):
        p = [r.randrange(rows) for _ in range(rows)]
        parents.copy_(torch.tensor(p, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        now, copies, _ = model(now, p, pages)
        for pool in old:
            for a, b in copies:
                pool[b] = pool[a]
        assert slots.tolist() == now and all(torch.equal(a, b) for a, b in zip(pools, old))
