"""gdn_page_plan and gdn_page_release against the definition, one request and token at a time, in
plain Python: whole numbers, equal everywhere."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as m
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    m.load_library()
    return m


def _i32(x):
    return torch.tensor(x, device="cuda", dtype=torch.int32)


def _clean(gdn):
    st = gdn.gdn_get_device_error()
    assert st == 0, gdn.gdn_status_string(st)


class Pool:
    """The pool as lists, and on the device."""

    def __init__(self, rows, columns, pages, page, seed=0):
        r = random.Random(seed)
        self.page, self.columns = page, columns
        self.table = [[7] * columns for _ in range(rows)]
        self.held = [0] * rows
        self.free = list(range(pages))
        r.shuffle(self.free)
        self.count = pages
        self.gpu = dict(table=_i32(self.table).reshape(rows, columns), held=_i32(self.held),
                        free_pages=_i32(self.free), free_count=_i32([pages]))

    def plan(self, rows, kv, new, capacity, offset, pages):
        """Slots, positions, cu_seqlens, kv_len_out; `pages` is changed in place."""
        b_all = range(len(kv))
        rows = list(b_all) if rows is None else rows
        live = [r >= 0 for r in rows]
        ok = all(not l or (r < len(self.held) and k >= 0 and n >= 0)
                 for l, r, k, n in zip(live, rows, kv, new))
        need = []
        if ok:
            want = [-(-(k + n) // self.page) for k, n in zip(kv, new)]
            ok = all(not l or w <= self.columns for l, w in zip(live, want))
            need = [max(0, w - self.held[r]) if l else 0 for l, r, w in zip(live, rows, want)]
            tokens = sum(n for l, n in zip(live, new) if l)
            ok = ok and sum(need) <= self.count and tokens <= capacity
        if not ok:
            return [-1] * capacity, [0] * capacity, [0] * (len(kv) + 1), None
        slots, positions, cu, out = [], [], [0], []
        for b in b_all:
            if not live[b]:
                out.append(-1)
                cu.append(cu[-1])
                continue
            r = rows[b]
            for _ in range(need[b]):
                self.count -= 1
                self.table[r][self.held[r]] = self.free[self.count]
                self.held[r] += 1
            if pages is not None:
                pages[b][:self.held[r]] = self.table[r][:self.held[r]]
            for i in range(kv[b], kv[b] + new[b]):
                slots.append(self.table[r][i // self.page] * self.page + i % self.page)
                positions.append(offset + i)
            cu.append(cu[-1] + new[b])
            out.append(kv[b] + new[b])
        pad = capacity - len(slots)
        return slots + [-1] * pad, positions + [0] * pad, cu, out

    def release(self, rows, keep):
        rows = list(range(len(keep))) if rows is None else rows
        if any(r >= len(self.held) or (r >= 0 and k < 0) for r, k in zip(rows, keep)):
            return False
        given = []
        for r, k in zip(rows, keep):
            if r < 0:
                continue
            keeps = min(self.held[r], -(-k // self.page))
            given += self.table[r][keeps:self.held[r]]
        if self.count + len(given) > len(self.free):
            return False
        for r, k in zip(rows, keep):
            if r >= 0:
                self.held[r] = min(self.held[r], -(-k // self.page))
        for page in reversed(given):
            self.free[self.count] = page
            self.count += 1
        return True

    def check(self):
        assert self.gpu["free_count"].tolist() == [self.count]
        assert self.gpu["held"].tolist() == self.held
        assert self.gpu["free_pages"].tolist() == self.free
        if self.table and self.columns:
            assert self.gpu["table"].tolist() == self.table


def _plan_both(gdn, pool, rows, kv, new, capacity, offset=0, outputs=True, **kw):
    b = len(kv)
    pages = [[-3] * pool.columns for _ in range(b)]
    t = dict(slots=_i32([5] * capacity), positions=_i32([5] * capacity),
             cu_seqlens=_i32([5] * (b + 1)), kv_len_out=_i32([5] * b),
             pages=_i32(pages).reshape(b, pool.columns))
    want = pool.plan(rows, kv, new, capacity, offset, pages)
    gdn.gdn_page_plan(_i32(kv), _i32(new), **(t if outputs else {}), **pool.gpu,
                      page_size=pool.page, rows=None if rows is None else _i32(rows),
                      position_offset=offset, **kw)
    if outputs:
        names = ("slots", "positions", "cu_seqlens", "kv_len_out")
        for name, x in zip(names, want):
            assert t[name].tolist() == ([5] * b if x is None else x), name
        if pool.columns and b:
            assert t["pages"].tolist() == pages
    pool.check()
    return want[3] is not None


@pytest.mark.parametrize("b,rows,columns,page,most", [
    (1, 1, 1, 16, 16), (1, 3, 700, 128, 50000), (7, 9, 40, 16, 300), (64, 64, 60, 64, 900),
    (513, 700, 9, 32, 60), (1500, 1500, 3, 128, 20), (8192, 8200, 2, 16, 6)])
def test_steps_of_a_server(gdn, b, rows, columns, page, most):
    """Steps in a row: new tokens for a batch in any order with entries left out, then what was
    not kept goes back, until requests end."""
    r = random.Random(b)
    pool = Pool(rows, columns, rows * columns, page, seed=b)
    length = [0] * rows
    for step in range(6 if b < 1000 else 3):
        at = r.sample(range(rows), b)
        at = [-1 if b > 1 and r.random() < 0.1 else x for x in at]
        kv = [length[x] if x >= 0 else r.choice([-5, 3]) for x in at]
        new = [min(r.choice([0, 1, r.randint(0, most)]), columns * page - k) if x >= 0 else -2
               for x, k in zip(at, kv)]
        capacity = sum(max(0, n) for n in new) + r.choice([0, 1, 77])
        assert _plan_both(gdn, pool, at, kv, new, capacity, offset=step * 1000)
        keep = [max(0, k + r.choice([0, n // 2, n, -k])) if x >= 0 else -1
                for x, k, n in zip(at, kv, new)]
        assert pool.release(at, keep)
        gdn.gdn_page_release(_i32(keep), **pool.gpu, page_size=page, rows=_i32(at))
        pool.check()
        for x, k in zip(at, keep):
            if x >= 0:
                length[x] = k
    _clean(gdn)
    everything = [h for h in pool.held]
    pool.release(list(range(rows))[:8192], [0] * min(rows, 8192))
    gdn.gdn_page_release(_i32([0] * min(rows, 8192)), **pool.gpu, page_size=page,
                         rows=_i32(list(range(rows))[:8192]))
    pool.check()
    assert sum(everything) + pool.count >= rows * columns
    _clean(gdn)


@pytest.mark.parametrize("columns", [1, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 127, 128, 129, 256, 257])
def test_tables_of_any_width(gdn, columns):
    """Block tables around the widths that share a warp, of one request and of many."""
    for b in (1, 3, 37, 130):
        test_steps_of_a_server(gdn, b, b + 2, columns, 16, 16 * columns // 3 + 1)


def test_what_was_taken_comes_back_as_it_was(gdn):
    pool = Pool(20, 30, 500, 16, seed=3)
    before = {k: x.clone() for k, x in pool.gpu.items()}
    kv = [0] * 20
    _plan_both(gdn, pool, None, kv, [100 + i for i in range(20)], 4000)
    pool.release(None, kv)
    gdn.gdn_page_release(_i32(kv), **pool.gpu, page_size=16)
    for k in ("held", "free_pages", "free_count"):
        assert torch.equal(pool.gpu[k], before[k])
    _clean(gdn)


def test_long_prompts(gdn):
    """240,000 tokens of a few requests, and one request over 100,000 columns."""
    pool = Pool(4, 6000, 24000, 16, seed=1)
    assert _plan_both(gdn, pool, [2, 0, 3], [5, 0, 17], [90000, 60000, 90000], 240000, offset=9)
    pool = Pool(1, 100000, 100003, 16, seed=2)
    assert _plan_both(gdn, pool, None, [0], [1000], 1000)
    assert _plan_both(gdn, pool, None, [1000], [1598000], 1598000)
    _clean(gdn)


ALL_OR_NOTHING = [
    dict(new=[17, 5, 200]),                              # more pages than are free
    dict(capacity=27),                                   # more tokens than there is room for
    dict(kv=[0, -1, 0]), dict(new=[4, -1, 4]), dict(rows=[0, 5, 1]),
    dict(rows=[0, 2 ** 31 - 1, 1]),
    dict(kv=[150, 0, 0], new=[20, 1, 1]),                # more pages than a row has
    dict(kv=[2 ** 31 - 1, 0, 0], new=[2 ** 31 - 1, 1, 1], capacity=100),
    dict(new=[2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]),
]


@pytest.mark.parametrize("bad", ALL_OR_NOTHING)
def test_all_or_nothing(gdn, bad):
    pool = Pool(5, 10, 12, 16, seed=4)
    case = {**dict(rows=[4, 0, 2], kv=[0, 0, 0], new=[10, 8, 10], capacity=28), **bad}
    assert not _plan_both(gdn, pool, case["rows"], case["kv"], case["new"], case["capacity"])
    assert gdn.gdn_get_device_error() == 6
    assert _plan_both(gdn, pool, [4, 0, 2], [0, 0, 0], [10, 8, 10], 28)
    _clean(gdn)
    assert not pool.release([4, 5, 2], [0, 0, 0]) and not pool.release([4, 0], [0, -1])
    for rows, keep in (([4, 5, 2], [0, 0, 0]), ([4, 0], [0, -1])):
        gdn.gdn_page_release(_i32(keep), **pool.gpu, page_size=16, rows=_i32(rows))
        assert gdn.gdn_get_device_error() == 6
        pool.check()


@pytest.mark.parametrize("count", [-1, 13, 2 ** 31 - 1])
def test_counts_out_of_range(gdn, count):
    """A pool whose counts are damaged is left alone: nothing is read or written by them."""
    for held in ([0, 0], [11, 0], [-1, 0], [2 ** 31 - 1, 1]):
        for free_count in (12, count):
            if held == [0, 0] and free_count == 12:
                continue
            pool = Pool(2, 10, 12, 16)
            pool.held, pool.count = held, free_count
            pool.gpu["held"].copy_(_i32(held))
            pool.gpu["free_count"].copy_(_i32([free_count]))
            slots = _i32([5] * 8)
            gdn.gdn_page_plan(_i32([0, 0]), _i32([4, 4]), slots, **pool.gpu, page_size=16)
            assert gdn.gdn_get_device_error() == 6 and slots.tolist() == [-1] * 8
            pool.check()
            gdn.gdn_page_release(_i32([0, 0]), **pool.gpu, page_size=16)
            assert gdn.gdn_get_device_error() == 6
            pool.check()


def test_damaged_page_ids(gdn):
    """A page id outside the pool gives slot -1 and is recorded."""
    pool = Pool(2, 4, 8, 16)
    pool.gpu["free_pages"][7] = 8                          # the first that is taken
    pool.gpu["free_pages"][6] = -1
    slots = _i32([5] * 40)
    gdn.gdn_page_plan(_i32([0, 0]), _i32([40, 0]), slots, **pool.gpu, page_size=16)
    assert gdn.gdn_get_device_error() == 6
    assert slots.tolist()[:32] == [-1] * 32
    assert slots.tolist()[32:] == [pool.free[5] * 16 + i for i in range(8)]


def test_few_outputs_in_place_and_empty(gdn):
    pool = Pool(3, 8, 20, 16, seed=6)
    kv, new = _i32([0, 3, 0]), _i32([20, 30, 0])
    assert pool.plan(None, [0, 3, 0], [20, 30, 0], 1 << 30, 0, None)
    gdn.gdn_page_plan(kv, new, kv_len_out=kv, **pool.gpu, page_size=16)   # in place, no slots
    assert kv.tolist() == [20, 33, 0]
    pool.check()
    positions = _i32([5] * 4)
    pool.plan(None, [20, 33, 0], [1, 1, 1], 4, 7, None)
    gdn.gdn_page_plan(kv, _i32([1, 1, 1]), positions=positions, **pool.gpu, page_size=16,
                      position_offset=7)
    assert positions.tolist() == [27, 40, 7, 0]
    pool.check()
    none = _i32([])
    slots, cu = _i32([5] * 3), _i32([5])
    gdn.gdn_page_plan(none, none, slots, cu_seqlens=cu, **pool.gpu, page_size=16)
    assert slots.tolist() == [-1] * 3 and cu.tolist() == [0]
    gdn.gdn_page_release(none, **pool.gpu, page_size=16)
    pool.check()
    _clean(gdn)


def test_captured_steps(gdn):
    """A plan and a release in one graph, replayed on a side stream as the lengths grow."""
    pool = Pool(6, 20, 120, 16, seed=9)
    length = [3, 0, 40, 17, 100, 1]
    pool.plan(None, [0] * 6, length, 1000, 0, None)
    gdn.gdn_page_plan(_i32([0] * 6), _i32(length), **pool.gpu, page_size=16)
    kv, new, kept = _i32(length), _i32([5] * 6), _i32([2] * 6)
    slots, positions, out = _i32([0] * 30), _i32([0] * 30), _i32([0] * 6)
    keep = _i32([0] * 6)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        gdn.gdn_page_plan(kv, new, slots, positions, kv_len_out=out, **pool.gpu, page_size=16)
        keep.copy_(kv + kept)
        gdn.gdn_page_release(keep, **pool.gpu, page_size=16)
        kv.copy_(keep)
    for _ in range(20):
        want = pool.plan(None, length, [5] * 6, 30, 0, None)
        pool.release(None, [x + 2 for x in length])
        length = [x + 2 for x in length]
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert slots.tolist() == want[0] and positions.tolist() == want[1]
        assert out.tolist() == want[3]
        pool.check()
    _clean(gdn)


def test_refusals(gdn):
    pool = Pool(2, 4, 8, 16)
    one, two = _i32([1]), _i32([1, 1])
    for bad in (dict(kv_len=two.long()), dict(new_len=one), dict(slots=two.long()),
                dict(slots=two, positions=one), dict(cu_seqlens=two), dict(kv_len_out=one),
                dict(pages=two), dict(rows=one), dict(rows=two.cpu()), dict(page_size=24),
                dict(held=one), dict(free_count=two), dict(table=pool.gpu["table"].t()),
                dict(free_pages=pool.gpu["table"]), dict(kv_len=_i32([1] * 3), new_len=_i32([1] * 3))):
        a = {**dict(kv_len=two, new_len=two, page_size=16), **pool.gpu, **bad}
        with pytest.raises((ValueError, TypeError, gdn.GDNError)):
            gdn.gdn_page_plan(a.pop("kv_len"), a.pop("new_len"), **a)
    with pytest.raises(ValueError):
        gdn.gdn_page_release(_i32([0] * 3), **pool.gpu, page_size=16)
    with pytest.raises(ValueError):
        gdn.gdn_page_release(two, **pool.gpu, page_size=16, rows=one)
    pool.check()
    _clean(gdn)
