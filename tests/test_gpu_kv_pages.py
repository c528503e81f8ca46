"""The pool of pages on the GPU (extend, free, fork, copy, compact) against a
plain Python bookkeeping: whole numbers and bytes, equal everywhere."""
import random

import pytest
import torch

from gqa_reference import Pool

dsa = pytest.importorskip("sparse_attention_logits_b200")

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """A pool on the GPU beside its plain form."""

    def __init__(self, batch, max_pages, page, num_pages, caches=((3, 16),), seed=0):
        self.plain = Pool(batch, max_pages, page, num_pages)
        self.page = page
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32, device="cuda")
        self.length = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.count = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.caches = [torch.randint(0, 255, (num_pages, *shape), generator=g, device="cuda").to(torch.uint8) for shape in caches]
        self.bytes = [c.clone() for c in self.caches]

    def moved(self, pairs):
        if pairs:
            src, dst = (list(x) for x in zip(*pairs))
            for c in self.bytes:
                c[dst] = c[src].clone()

    def same(self):
        assert self.length.tolist() == self.plain.length
        assert self.count.tolist() == self.plain.count
        assert self.table.tolist() == self.plain.table
        for a, b in zip(self.caches, self.bytes):
            assert torch.equal(a, b)

    def extend(self, seqs, add):
        dsa.kv_pages_extend(self.table, self.length, self.count, _i32(seqs), _i32(add), self.page)
        return self.plain.extend(seqs, add)

    def free(self, seqs):
        dsa.kv_pages_free(self.table, self.length, self.count, _i32(seqs), self.page)
        self.plain.free(seqs)

    def fork(self, parents, children):
        dsa.kv_pages_fork(self.table, self.length, self.count, _i32(parents), _i32(children), self.page, self.caches)
        self.moved(self.plain.fork(parents, children))

    def compact(self, in_place):
        if in_place:
            dsa.kv_pages_compact(self.table, self.count, self.caches, table_out=self.table, ref_out=self.count)
        else:
            t, c = self.table.clone(), self.count.clone()
            self.table, self.count = dsa.kv_pages_compact(self.table, self.count, self.caches)
            assert t.tolist() == self.plain.table and c.tolist() == self.plain.count
        self.moved(self.plain.compact())


# (batch, table width, page size, pool, caches' page shapes)
POOLS = {
    "small": (6, 5, 4, 20, ((3, 16),)),
    "page_of_1": (8, 40, 1, 100, ((16,), (32,))),
    "one_page_pool": (2, 3, 8, 1, ((16,),)),
    "odd_sizes": (17, 9, 7, 101, ((5, 16), (1, 48), (7, 4096))),
    "many_pages": (40, 300, 16, 9000, ((64,),)),
    "large_pages": (12, 6, 16, 50, ((2, 16, 1024), (80016,))),
    "no_caches": (5, 6, 3, 33, ()),
}


@pytest.mark.parametrize("case", list(POOLS))
@pytest.mark.parametrize("seed", [0, 1])
def test_random_lives(cuda_device, case, seed):
    """Sequences admitted, grown, branched, dropped and the pool compacted at random, many rounds."""
    batch, width, page, pages, caches = POOLS[case]
    r = random.Random(seed * 1000 + len(case))
    p = Both(batch, width, page, pages, caches, seed)
    refused = False
    for _ in range(25):
        act = r.choice(["extend", "extend", "free", "fork", "fork", "compact"])
        some = r.sample(range(batch), r.randint(1, batch))
        if act == "extend":
            add = [r.choice([0, 1, r.randint(1, page * width)]) for _ in some]
            refused |= not p.extend(some, add)
        elif act == "free":
            p.free(some[:max(1, len(some) // 2)] + [-1])
        elif act == "fork":
            empty = [q for q in range(batch) if p.plain.length[q] == 0]
            full = [q for q in range(batch) if p.plain.length[q] > 0]
            if not empty or not full:
                continue
            children = r.sample(empty, r.randint(1, len(empty)))
            p.fork([r.choice(full) for _ in children] + [0], children + [-1])
        else:
            p.compact(r.random() < 0.5)
        p.same()
    st = dsa._lib.dsa_get_device_error(torch.cuda.current_stream().cuda_stream)
    assert st in (dsa.DSA_OK, dsa.DSA_ERR_OUT_OF_PAGES, dsa.DSA_ERR_INVALID_ARG)    # some rounds ask for too much


def test_lowest_pages_first_in_list_order(cuda_device):
    p = Both(4, 4, 4, 12)
    p.extend([3, 0, -1, 2], [5, 4, 9, 13])
    assert p.table.tolist() == [[2, -1, -1, -1], [-1] * 4, [3, 4, 5, 6], [0, 1, -1, -1]]
    p.free([0])
    p.extend([1], [1])                              # the freed page is the lowest
    assert p.table[1].tolist() == [2, -1, -1, -1]
    p.same()
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK


def _status():
    return dsa._lib.dsa_get_device_error(torch.cuda.current_stream().cuda_stream)


def test_want_of_pages_leaves_a_sequence_as_it_was(cuda_device):
    p = Both(4, 8, 4, 5)
    p.extend([0, 1, 2], [8, 16, 4])                 # 2 + 4 + 1 pages of 5: the second does not fit, nor the third behind it
    assert _status() == dsa.DSA_ERR_OUT_OF_PAGES
    assert p.length.tolist() == [8, 0, 0, 0]
    p.same()
    p.extend([1, 0], [11, 0])                       # 3 pages: exactly the rest
    assert _status() == dsa.DSA_OK
    p.fork([1], [3])                                # its last page needs a copy: none left
    assert _status() == dsa.DSA_ERR_OUT_OF_PAGES
    p.fork([0], [3])                                # full pages only: nothing fresh needed
    assert _status() == dsa.DSA_OK
    p.same()


def test_bad_entries_are_reported_and_change_nothing(cuda_device):
    p = Both(3, 4, 4, 12)
    p.extend([0, 1], [6, 3])
    for seqs, add in (([3], [1]), ([-2], [1]), ([2], [17]), ([2], [-1]), ([0], [11])):
        p.extend(seqs, add) if seqs[0] >= 0 else dsa.kv_pages_extend(p.table, p.length, p.count, _i32(seqs), _i32(add), 4)
        assert _status() == dsa.DSA_ERR_INVALID_ARG, (seqs, add)
        p.same()
    p.extend([2, 2], [3, 5])                        # listed twice: the first counts
    assert _status() == dsa.DSA_ERR_INVALID_ARG
    p.same()
    for parents, children in (([0], [1]), ([0], [3]), ([5], [2]), ([-1], [2])):
        dsa.kv_pages_fork(p.table, p.length, p.count, _i32(parents), _i32(children), 4, p.caches)
        assert _status() == dsa.DSA_ERR_INVALID_ARG, (parents, children)
        p.same()
    dsa.kv_pages_free(p.table, p.length, p.count, _i32([7]), 4)
    assert _status() == dsa.DSA_ERR_INVALID_ARG
    p.free([2, 2])                                  # listed twice: freed once
    assert _status() == dsa.DSA_OK
    p.same()
    p.fork([0, 1, 0], [2, 2, 2])                    # one child three times: the first counts
    assert _status() == dsa.DSA_ERR_INVALID_ARG
    p.same()


def test_fork_of_an_empty_sequence_and_of_itself(cuda_device):
    p = Both(4, 4, 4, 12)
    p.extend([0], [5])
    p.fork([1, 2, 0], [2, 3, 1])                    # 2 and 3 branch off sequences empty at the start: stay empty
    assert _status() == dsa.DSA_OK
    p.same()
    assert p.length.tolist() == [5, 5, 0, 0]


@pytest.mark.parametrize("n_caches", [1, 3, 97, 200])
def test_copy(cuda_device, n_caches):
    """Pairs in every cache, of several page sizes; unused pairs and pairs to themselves skipped."""
    g = torch.Generator(device="cuda").manual_seed(9)
    sizes = [16, 48, 4096, 16400, 40000]
    caches = [torch.randint(0, 255, (23, sizes[i % 5]), generator=g, device="cuda").to(torch.uint8) for i in range(n_caches)]
    want = [c.clone() for c in caches]
    src, dst = [0, 5, -1, 7, 3, 2], [10, 11, 12, -1, 3, 22]
    dsa.kv_pages_copy(caches, _i32(src), _i32(dst))
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    for c, w in zip(caches, want):
        for a, b in ((0, 10), (5, 11), (2, 22)):
            w[b] = w[a].clone()
        assert torch.equal(c, w)
    dsa.kv_pages_copy(caches, _i32([23, 1, 1]), _i32([1, -7, 2]))
    assert _status() == dsa.DSA_ERR_INVALID_ARG
    for c, w in zip(caches, want):
        w[2] = w[1].clone()
        assert torch.equal(c, w)


def test_large_pool_and_long_lists(cuda_device):
    """More pages than one pass of a block covers, lists longer than a block, in order."""
    batch, width, page, pages = 2500, 40, 2, 70001
    r = random.Random(4)
    p = Both(batch, width, page, pages, ())
    order = r.sample(range(batch), batch)
    p.extend(order, [r.randint(0, 60) for _ in order])
    p.free(r.sample(range(batch), 1200))
    empty = [q for q in range(batch) if p.plain.length[q] == 0]
    full = [q for q in range(batch) if p.plain.length[q] > 0]
    p.fork([r.choice(full) for _ in empty], empty)
    p.compact(True)
    p.free(r.sample(range(batch), 1200))
    p.compact(False)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    p.same()


def test_largest_pool_and_list(cuda_device):
    """As many pages and list entries as a call takes: the books fill the cluster's shared memory."""
    n, pages, page = 4096, 1 << 22, 4
    r = random.Random(5)
    p = Both(2 * n, 9, page, pages, ())
    held = torch.arange(0, pages, 3, device="cuda")         # a third of the pool is someone else's
    p.count[held] = 1
    for i in held.tolist():
        p.plain.count[i] = 1
    p.extend(r.sample(range(n), n), [r.randint(0, 9 * page) for _ in range(n)])
    p.fork([r.randrange(n) for _ in range(n)], r.sample(range(n, 2 * n), n))
    assert _status() == dsa.DSA_OK
    p.same()
    p.free(list(range(n)))
    p.compact(True)
    assert _status() == dsa.DSA_OK
    p.same()
    with pytest.raises(dsa.DSAError):
        dsa.kv_pages_free(p.table, p.length, p.count, _i32([0] * (n + 1)), page)


def test_captured_turnover(cuda_device):
    """free + extend + fork captured once and replayed: the books follow without a host read."""
    p = Both(6, 8, 4, 40, ((32,),))
    p.extend([0, 1, 2], [9, 13, 30])
    gone, grow, add = _i32([0, 1]), _i32([0, 1]), _i32([5, 7])
    par, child = _i32([2]), _i32([4])

    def turn():
        dsa.kv_pages_free(p.table, p.length, p.count, gone, 4)
        dsa.kv_pages_extend(p.table, p.length, p.count, grow, add, 4)
        dsa.kv_pages_free(p.table, p.length, p.count, child, 4)
        dsa.kv_pages_fork(p.table, p.length, p.count, par, child, 4, p.caches)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        turn()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    for lists in (None, ([0, 1], [0, 1], [5, 7]), ([1, -1], [3, 1], [11, 2]), ([3, 0], [0, 3], [1, 1])):
        if lists:
            for t, x in zip((gone, grow, add), lists):
                t.copy_(_i32(x))
            graph.replay()
        p.plain.free(gone.tolist())
        p.plain.extend(grow.tolist(), add.tolist())
        p.plain.free([4])
        p.moved(p.plain.fork([2], [4]))
        p.same()
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK


def _pool_of(lens, page, width, num_pages):
    """Books for sequences of these lengths, extended in one call."""
    p = Both(len(lens) + 2, width, page, num_pages, ((page * 16,),))
    p.extend(list(range(len(lens))), lens)
    assert _status() == dsa.DSA_OK
    p.same()
    return p


@pytest.mark.parametrize("at,bad", [(0, -1), (1, 12), (1, 10 ** 6), (2, -1), (2, -7), (2, 12)])
@pytest.mark.parametrize("tail", [1, 4])
def test_fork_of_a_parent_with_a_bad_page_changes_nothing(cuda_device, tail, at, bad):
    """A parent one of whose pages (a full one, or the last) is out of range: its branch is refused whole, the others of
    the same call are served, and a page that the refused one would have taken goes to the next."""
    p = _pool_of([8 + tail, 7], 4, 4, 12)               # parent 0: two full pages and one of `tail` tokens
    was = int(p.table[0, at])
    p.table[0, at] = bad
    before = [x.clone() for x in (p.table, p.length, p.count, *p.caches)]
    dsa.kv_pages_fork(p.table, p.length, p.count, _i32([0]), _i32([2]), 4, p.caches)
    assert _status() == dsa.DSA_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(before, (p.table, p.length, p.count, *p.caches)))
    dsa.kv_pages_fork(p.table, p.length, p.count, _i32([0, 1]), _i32([2, 3]), 4, p.caches)
    assert _status() == dsa.DSA_ERR_INVALID_ARG
    p.table[0, at] = was
    p.moved(p.plain.fork([1], [3]))
    p.same()


def test_many_forks_with_bad_pages_among_them(cuda_device):
    """More entries than the cluster's blocks have warps, every seventh parent with a page out of range."""
    n, page, width = 600, 4, 70
    r = random.Random(6)
    lens = [r.randint(1, page * width) for _ in range(n)]
    p = Both(2 * n, width, page, sum(-(-x // page) for x in lens) + n, ())
    p.extend(list(range(n)), lens)
    kept = p.table.clone()
    for q in range(0, n, 7):
        p.table[q, r.randrange(-(-lens[q] // page))] = r.choice([-1, -3, p.count.numel(), 2 ** 31 - 1])
    broken = p.table.clone()
    dsa.kv_pages_fork(p.table, p.length, p.count, _i32(list(range(n))), _i32(list(range(n, 2 * n))), page, ())
    assert _status() == dsa.DSA_ERR_INVALID_ARG
    assert torch.equal(p.table[:n], broken[:n])
    p.table[:n] = kept[:n]
    good = [q for q in range(n) if q % 7]
    p.plain.fork(good, [n + q for q in good])
    p.same()


@pytest.mark.parametrize("bad", [-1, -5, 12, 2 ** 31 - 1])
def test_free_of_a_sequence_with_a_bad_page(cuda_device, bad):
    """Dropped all the same: the page out of range is passed over and reported, the others are given back."""
    p = _pool_of([9, 7], 4, 4, 12)
    page = int(p.table[0, 1])
    p.table[0, 1] = bad
    dsa.kv_pages_free(p.table, p.length, p.count, _i32([0]), 4)
    assert _status() == dsa.DSA_ERR_INVALID_ARG
    p.plain.free([0])
    p.plain.count[page] = 1                                 # nobody's any more, and not given back
    p.same()


@pytest.mark.parametrize("seed", [2, 3, 4])
def test_random_lives_report_what_was_refused(cuda_device, seed):
    """After each action the device status is the one that the plain books give: entries out of range first, then
    want of pages, else none."""
    batch, width, page, pages = 12, 6, 4, 14
    r = random.Random(seed)
    p = Both(batch, width, page, pages, ((16,),), seed)
    met = set()
    for _ in range(60):
        act, some = r.choice(["extend", "extend", "free", "fork"]), r.sample(range(batch), r.randint(1, 3))
        free, length = p.plain.count.count(0), list(p.plain.length)
        asked, invalid, short = 0, False, False

        def want(n):
            nonlocal asked, short
            asked += n
            short |= n > 0 and asked > free
        if act == "extend":
            add = [-1 if r.random() < 0.1 else r.randint(0, page * width) for _ in some]
            for q, a in zip(some, add):
                if a < 0 or length[q] + a > page * width:
                    invalid = True
                else:
                    want(p.plain.up(length[q] + a) - p.plain.up(length[q]))
            p.extend(some, add)
        elif act == "free":
            p.free(some)
        else:
            parents = [r.randrange(batch) for _ in some]
            for a, b in zip(parents, some):
                if length[b]:
                    invalid = True
                else:
                    want(length[a] % page > 0)
            p.fork(parents, some)
        code = dsa.DSA_ERR_INVALID_ARG if invalid else dsa.DSA_ERR_OUT_OF_PAGES if short else dsa.DSA_OK
        met.add(code)
        assert _status() == code, act
        p.same()
    assert len(met) == 3


@pytest.mark.parametrize("dtype,d,heads", [(torch.bfloat16, 576, 128), (torch.float32, 64, 8)])
def test_pool_serves_the_latent_cache_of_sparse_attention(cuda_device, dtype, d, heads):
    """dsa_sparse_mla over pages that the pool handed out, branched and drew together, against the same rows in a
    contiguous cache (a table as wide as the context, -1 behind each sequence)."""
    g = torch.Generator(device="cuda").manual_seed(11)
    page, ctx, batch, pages, d_v = 64, 512, 3, 24, 512 if d == 576 else d
    table = torch.full((batch, ctx // page), -1, dtype=torch.int32, device="cuda")
    length, count = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    cache = torch.zeros((pages, page, d), dtype=dtype, device="cuda")
    whole = torch.randn((batch, ctx, d), generator=g, device="cuda").to(dtype)
    count[[0, 2, 5, 9]] = 1                                 # pages held by someone else
    lens = [200, 300]
    dsa.kv_pages_extend(table, length, count, _i32([0, 1]), _i32(lens), page)
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            cache[int(table[b, j]), :min(page, n - j * page)] = whole[b, j * page:min(n, (j + 1) * page)]
    dsa.kv_pages_fork(table, length, count, _i32([1]), _i32([2]), page, [cache])
    whole[2, :lens[1]] = whole[1, :lens[1]]
    lens.append(lens[1])
    count[[0, 2, 5, 9]] = 0
    dsa.kv_pages_compact(table, count, [cache], table_out=table, ref_out=count)
    dsa.kv_pages_extend(table, length, count, _i32([2]), _i32([1]), page)
    lens[2] += 1
    cache[int(table[2, 300 // page]), 300 % page] = whole[2, 300]
    idx = torch.full((batch, 256), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        some = torch.randperm(n - 1)[:min(n - 1, 255)].to(torch.int32)
        idx[b, :len(some)] = some
        idx[b, len(some)] = n - 1
    idx, rows = idx.cuda(), _i32([0, 1, 2])
    q = torch.randn((batch, heads, d), generator=g, device="cuda").to(dtype)
    out, lse = dsa.sparse_mla(q, cache, idx, rows, 0.05, d_v, ctx, page_table=table)
    ref, ref_lse = dsa.sparse_mla(q, whole, idx, rows, 0.05, d_v, ctx)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
