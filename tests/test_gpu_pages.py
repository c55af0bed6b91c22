"""Pages of a cache on the GPU against a page-by-page model on the host; every result is exact."""
from __future__ import annotations

import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from prefix_scan_gb300 import PrefixScanError, api  # noqa: E402

DEV = torch.device("cuda:0")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Model:
    """The same operations on lists: pages hold a number that says which page's data they have."""

    def __init__(self, pages, rows, width, page_tokens, seed, fill=0.6):
        r = random.Random(seed)
        self.pages, self.width, self.pt, self.r = pages, width, page_tokens, r
        free = list(range(pages))
        r.shuffle(free)
        self.table, self.lengths, self.ref = [], [], [0] * pages
        left = int(fill * pages)
        for _ in range(rows):
            n = min(r.randrange(0, width + 1), left)
            left -= n
            row = [free.pop() for _ in range(n)]
            self.lengths.append(max(0, n * page_tokens - r.choice([0, r.randrange(page_tokens)])) if n else 0)
            for p in row:
                self.ref[p] += 1
            self.table.append(row + [-1] * (width - n))
        self.data = list(range(pages))

    def gpu(self, elems, dtypes):
        self.pools0 = [torch.randint(-100, 100, (self.pages, e), device=DEV).to(d) for e, d in zip(elems, dtypes)]
        return (ints(self.table).view(len(self.table), self.width), ints(self.lengths), ints(self.ref),
                [p.clone() for p in self.pools0])

    def free_pages(self):
        return [p for p in range(self.pages) if self.ref[p] <= 0]

    def fork(self, parents):
        free, new, lens, missing = iter(self.free_pages()), [], [], 0
        refs = list(self.ref)
        for p in parents:
            if not 0 <= p < len(self.table):
                new.append([-1] * self.width)
                lens.append(0)
                continue
            n = min(max(self.lengths[p], 0), self.width * self.pt)
            row = [-1] * self.width
            for j in range(n // self.pt):
                q = self.table[p][j]
                if 0 <= q < self.pages:
                    row[j] = q
                    refs[q] += 1
            old = self.table[p][n // self.pt] if n % self.pt else -1
            if 0 <= old < self.pages:
                q = next(free, -1)
                row[n // self.pt] = q
                if q < 0:
                    missing += 1
                else:
                    refs[q] += 1
                    self.data[q] = self.data[old]
            new.append(row)
            lens.append(n)
        self.ref = refs
        return new, lens, missing

    def grow(self, table, lengths, new_lengths):
        free, missing = iter(self.free_pages()), 0
        given = []
        for row, a, b in zip(table, lengths, new_lengths):
            a = min(max(a, 0), self.width * self.pt)
            for j in range(-(-a // self.pt), -(-max(b, 0) // self.pt)):
                if j >= self.width:
                    missing += 1
                elif not 0 <= row[j] < self.pages:
                    row[j] = next(free, -1)
                    missing += row[j] < 0
                    given.append(row[j])
        for p in given:
            if p >= 0:
                self.ref[p] = 1
        return missing

    def drop(self, table, flags):
        for row, f in zip(table, flags):
            if f:
                for p in row:
                    if 0 <= p < self.pages:
                        self.ref[p] -= 1
                row[:] = [-1] * self.width

    def compact(self):
        used = [p for p in range(self.pages) if self.ref[p] > 0]
        m = len(used)
        to = {p: p for p in used if p < m}
        for p, h in zip([p for p in used if p >= m], [p for p in range(m) if self.ref[p] <= 0]):
            to[p] = h
            self.data[h] = self.data[p]
            self.ref[h], self.ref[p] = self.ref[p], 0
        self.table = [[to.get(p, -1) for p in row] for row in self.table]
        return m

    def check(self, ref, pools, **pairs):
        torch.cuda.synchronize()
        assert ref.tolist() == self.ref
        for now, was in zip(pools, self.pools0):
            assert torch.equal(now, was[torch.tensor(self.data, device=DEV)])
        for name, (got, want) in pairs.items():
            assert got.tolist() == want, name


POOLS = [([5], [torch.int8]), ([2048, 16384], [torch.bfloat16, torch.float32]), ([3, 1000, 8], [torch.int32, torch.int16, torch.int64])]


@pytest.mark.parametrize("elems,dtypes", POOLS)
@pytest.mark.parametrize("pages,rows,width,pt", [(1, 1, 1, 1), (40, 5, 4, 16), (300, 17, 9, 7), (2000, 64, 20, 1), (500, 3, 70, 1 << 24)])
def test_fork_grow_free_compact(pages, rows, width, pt, elems, dtypes):
    m = Model(pages, rows, width, pt, pages)
    table, lengths, ref, pools = m.gpu(elems, dtypes)
    parents = [m.r.randrange(-1, rows + 1) for _ in range(2 * rows + 1)]
    new, lens, missing = m.fork(parents)
    t2, l2, miss = api.pages_fork(table, lengths, ints(parents), ref, pools, page_tokens=pt)
    m.check(ref, pools, table=(t2, new), lengths=(l2, lens), missing=(miss, [missing]))
    more = [n + m.r.randrange(-1, 3) * pt + m.r.randrange(2) for n in lens]
    more = [min(n, 2 ** 31 - 1) for n in more]
    missing = m.grow(new, lens, more)
    miss = api.pages_grow(t2, l2, ints(more), ref, page_tokens=pt)
    m.check(ref, pools, table=(t2, new), missing=(miss, [missing]))
    flags = [m.r.randrange(2) for _ in range(rows)]
    m.drop(m.table, flags)
    api.pages_free(table, ref, flags=torch.tensor(flags, dtype=torch.uint8, device=DEV))
    m.check(ref, pools, table=(table, m.table))
    both = torch.cat([table, t2])
    m.table = m.table + new
    used = m.compact()
    got = api.pages_compact(both, ref, pools)
    m.check(ref, pools, table=(both, m.table), used=(got, [used]))
    got = api.pages_compact(both, ref, pools)   # nothing left to move
    m.check(ref, pools, table=(both, m.table), used=(got, [used]))
    m.drop(m.table, [1] * len(m.table))
    api.pages_free(both, ref)
    m.check(ref, pools, table=(both, m.table))
    assert all(n == 0 for n in m.ref)


@pytest.mark.parametrize("pages", [16383, 16384, 16385, 70001])
def test_pools_past_a_tile_of_the_plan(pages):
    # the plans scan counts 16384 at a time: free pages, and the boundary m, on either side of a tile's end
    for fill in (0.02, 0.5, 0.98):
        m = Model(pages, pages // 50, 100, 3, pages, fill)
        table, lengths, ref, pools = m.gpu([1], [torch.int32])
        parents = [m.r.randrange(len(m.table)) for _ in range(700)]
        new, lens, missing = m.fork(parents)
        t2, _, miss = api.pages_fork(table, lengths, ints(parents), ref, pools, page_tokens=3)
        m.check(ref, pools, table=(t2, new), missing=(miss, [missing]))
        m.drop(new, [1] * 700)
        api.pages_free(t2, ref)
        used = m.compact()
        got = api.pages_compact(table, ref, pools)
        m.check(ref, pools, table=(table, m.table), used=(got, [used]))


def test_shared_pages_and_full_pool():
    # no free page: whole pages are still shared, last ones are missing
    table, lengths = ints([[0, 1], [2, -1]]), ints([6, 2])
    ref, pool = ints([1, 1, 1]), torch.arange(3, device=DEV)
    t2, l2, miss = api.pages_fork(table, lengths, ints([0, 0, 1]), ref, pool, page_tokens=4)
    assert t2.tolist() == [[0, -1], [0, -1], [-1, -1]] and l2.tolist() == [6, 6, 2]
    assert miss.item() == 3 and ref.tolist() == [3, 1, 1]
    miss = api.pages_grow(t2, l2, ints([9, 6, 2]), ref, page_tokens=4)
    assert miss.item() == 1 and t2.tolist() == [[0, -1], [0, -1], [-1, -1]]


def test_indices_out_of_range_are_none():
    table, lengths = ints([[7, -3, 1], [1 << 30, 0, 2]]), ints([-5, 1 << 30])
    ref, pool = ints([1, 1, 1, 0]), torch.arange(4, device=DEV, dtype=torch.int32)
    t2, l2, miss = api.pages_fork(table, lengths, ints([0, 1]), ref, pool, page_tokens=2)
    assert t2.tolist() == [[-1, -1, -1], [-1, 0, 2]] and l2.tolist() == [0, 6] and ref.tolist() == [2, 1, 2, 0]
    api.pages_free(table, ref)
    assert ref.tolist() == [1, 0, 1, 0] and (table == -1).all()
    api.pages_copy(pool, ints([0, 9, -1, 1]), ints([3, 0, 1, 4]))
    assert pool.tolist() == [0, 1, 2, 0]


def test_compact_forgets_entries_of_free_pages():
    # row 1's pages were freed elsewhere: its entries must not name what moves into their place
    table, ref = ints([[5, 4], [0, 3]]), ints([0, 1, 0, 0, 2, 1])
    pool = torch.arange(6, device=DEV).float()
    used = api.pages_compact(table, ref, pool)
    assert used.item() == 3 and table.tolist() == [[2, 0], [-1, -1]]
    assert ref.tolist() == [2, 1, 1, 0, 0, 0] and pool[:3].tolist() == [4, 1, 5]


@pytest.mark.parametrize("n", [0, 1, 37, 900])
def test_copy(n):
    pools = [torch.randn(2000, e, device=DEV) for e in (4, 4100, 33)]
    was = [p.clone() for p in pools]
    perm = torch.randperm(2000, device=DEV).to(torch.int32)
    src, dst = perm[:n].clone(), perm[1000:1000 + n].clone()
    api.pages_copy(pools, src, dst)
    for p, w in zip(pools, was):
        w[dst.long()] = w[src.long()]
        assert torch.equal(p, w)


def test_offsets_past_32_bits():
    # a pool of over 4 GiB: the last page moves to the front
    pages, elems = 70000, 16384
    pool = torch.zeros(pages, elems, dtype=torch.float32, device=DEV)
    pool[-1], pool[-2] = 3.0, 4.0
    ref = torch.zeros(pages, dtype=torch.int32, device=DEV)
    ref[-2:] = 1
    table = ints([[pages - 1, pages - 2]])
    used = api.pages_compact(table, ref, pool)
    assert used.item() == 2 and table.tolist() == [[1, 0]]
    assert (pool[0] == 4).all() and (pool[1] == 3).all()
    api.pages_copy(pool, ints([0]), ints([pages - 1]))
    assert (pool[-1] == 4).all()


def test_empty():
    none = ints([]).view(0, 4)
    ref, pool = ints([0, 0]), torch.zeros(2, 3, device=DEV)
    t, n, miss = api.pages_fork(none, ints([]), ints([]), ref, pool, page_tokens=4)
    assert t.shape == (0, 4) and miss.item() == 0
    t, n, miss = api.pages_fork(none, ints([]), ints([0, 5]), ref, pool, page_tokens=4)
    assert (t == -1).all() and n.tolist() == [0, 0]
    assert api.pages_grow(none, ints([]), ints([]), ref, page_tokens=4).item() == 0
    api.pages_free(none, ref)
    assert api.pages_compact(none, ref, pool).item() == 0
    assert api.pages_compact(none, ints([]), []).item() == 0


def test_another_stream_and_graph():
    m = Model(100, 8, 6, 5, 3)
    table, lengths, ref, pools = m.gpu([64], [torch.float32])
    parents = ints([1, 2, 3])
    ws = torch.empty(api.pages_workspace_size(8, 100), dtype=torch.uint8, device=DEV)
    t2, l2 = torch.empty(3, 6, dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        api.pages_fork(table, lengths, parents, ref, pools, page_tokens=5, out_table=t2, out_lengths=l2, workspace=ws)
    for _ in range(3):   # three forks, each on what the last one left
        new, lens, _ = m.fork([1, 2, 3])
        graph.replay()
        m.check(ref, pools, table=(t2, new), lengths=(l2, lens))


def test_step_on_forked_states():
    # two branches of one state take different tokens: the parent's state and the other branch stay as they are
    hv, k, v = 2, 64, 64
    pool = torch.randn(6, hv, k, v, device=DEV)
    was = pool.clone()
    table, ref = ints([[4]]), ints([0, 0, 0, 0, 1, 0])
    t2, _, _ = api.pages_fork(table, ints([10]), ints([0, 0]), ref, pool, page_tokens=1 << 30)
    assert t2.tolist() == [[0], [1]] and ref.tolist() == [1, 1, 0, 0, 1, 0]
    x = [torch.randn(2, 1, hv, n, device=DEV) for n in (k, k, v)] + [-torch.rand(2, 1, hv, device=DEV), torch.rand(2, 1, hv, device=DEV)]
    api.delta_rule_step(*x, pool, slots=t2[:, 0].contiguous())
    assert torch.equal(pool[2:], was[2:]) and not torch.equal(pool[0], pool[1])
    one = was[4:5].clone()
    api.delta_rule_step(*(t[1:] for t in x), one)
    assert torch.equal(pool[1], one[0])


def test_refusals():
    table, lengths, ref, pool = ints([[0]]), ints([1]), ints([1, 0]), torch.zeros(2, 4, device=DEV)
    with pytest.raises(ValueError, match="table"):
        api.pages_fork(table.long(), lengths, ints([0]), ref, pool, page_tokens=4)
    with pytest.raises(ValueError, match="length"):
        api.pages_fork(table, ints([1, 2]), ints([0]), ref, pool, page_tokens=4)
    with pytest.raises(ValueError, match="page_tokens"):
        api.pages_grow(table, lengths, lengths, ref, page_tokens=0)
    with pytest.raises(ValueError, match="pools"):
        api.pages_compact(table, ref, pool[:1])
    with pytest.raises(ValueError, match="pools"):
        api.pages_compact(table, ref, torch.zeros(4, 2, device=DEV).t())
    with pytest.raises(ValueError, match="flags"):
        api.pages_free(table, ref, flags=ints([1]))
    with pytest.raises(ValueError, match="workspace"):
        api.pages_compact(table, ref, pool, workspace=torch.empty(4, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="differ"):
        api.pages_copy(pool, ints([0]), ints([0, 1]))
    with pytest.raises(PrefixScanError, match="OVERLAP"):
        api.pages_fork(table, lengths, ints([0]), ref, pool, page_tokens=4, out_table=table)
    with pytest.raises(PrefixScanError, match="OVERLAP"):
        api.pages_compact(table, ref, [pool, pool])
