"""wenc_kv_extend and wenc_kv_release against plain loops over the sequences: whole numbers, so equal."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _t(a):
    import torch
    return torch.tensor(np.asarray(a, np.int32), dtype=torch.int32, device="cuda")


class Cache:
    """Tables and free pages of sequences with these lengths, on the host."""

    def __init__(self, lens, page, width, extra, seed, held=None):
        r = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        total = sum(need) + extra
        order = r.permutation(total).astype(np.int32)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            keep = range(n) if held is None else [e for e in range(n) if held(s, e)]
            for e in keep:
                self.table[s, e] = order[at]
                at += 1
        self.free = np.full(total, -1, np.int32)
        self.count = total - at
        self.free[:self.count] = order[at:]
        self.lens, self.page = list(lens), page


def _extend(c, new, rows, lens=None, **kw):
    import torch
    from transformer_encoder_gb300 import kv_extend
    table = kw.pop("table", None)
    if table is None:
        table = torch.from_numpy(c.table).cuda()
    free = torch.from_numpy(c.free).cuda()
    got = kv_extend(_t(new), _t(c.lens if lens is None else lens), table, free, _t([c.count]), c.page, rows, **kw)
    assert np.array_equal(free.cpu().numpy(), c.free)
    return table, got


def _want(c, new, rows):
    table, count, pos, slots = c.table.copy(), c.count, [], []
    for s, (m, n) in enumerate(zip(new, c.lens)):
        for e in range(-(-n // c.page), -(-(n + m) // c.page)):
            count -= 1
            table[s, e] = c.free[count]
        for p in range(n, n + m):
            pos.append(p)
            slots.append(int(table[s, p // c.page]) * c.page + p % c.page)
    pad = rows - len(pos)
    return table, [a + b for a, b in zip(new, c.lens)], count, np.cumsum([0] + list(new)), pos + [0] * pad, slots + [-1] * pad


@pytest.mark.parametrize("n,most,past,page,pad", [
    (1, 1, 0, 16, 0), (1, 1, 16, 16, 1), (3, 2, 5, 1, 0), (7, 40, 100, 16, 5), (256, 1, 500, 16, 0), (33, 600, 50, 24, 3),
    (513, 9, 33, 8, 100), (2047, 3, 10, 16, 2), (2049, 20, 100, 64, 1), (5000, 2, 4, 3, 0), (2, 9000, 3, 5, 7), (512, 3, 40, 16, 1),
    (2048, 1, 40, 16, 0), (9000, 1, 4, 8, 0), (9000, 0, 4, 8, 9), (20000, 1, 30, 16, 3)])
def test_extend(n, most, past, page, pad):
    from transformer_encoder_gb300 import sync_status
    r = np.random.default_rng(n + most)
    new, lens = r.integers(0, most + 1, n).tolist(), r.integers(0, past + 1, n).tolist()
    new[-1] = most
    width = -(-(most + past) // page) + 2
    c = Cache(lens, page, width, sum(-(-m // page) + 1 for m in new) + 2, n)
    rows = sum(new) + pad
    table, (lens2, count, start, pos, slots) = _extend(c, new, rows)
    sync_status()
    want = _want(c, new, rows)
    for got, w in zip((table, lens2, count, start, pos, slots), want):
        assert np.array_equal(got.cpu().numpy().ravel(), np.asarray(w).ravel())


def test_extend_takes_the_last_page_and_no_more():
    import torch
    from transformer_encoder_gb300 import WencError, sync_status
    c = Cache([15, 16, 3], 16, 6, 0, 1)
    c.free = np.concatenate([c.free, [90, 91]]).astype(np.int32)
    c.free[:2], c.count = [90, 91], 2
    new = [2, 16, 0]
    table, got = _extend(c, new, 20)
    sync_status()
    assert got[1].item() == 0 and table[0, 1].item() == 91 and table[1, 1].item() == 90
    # one page too few: nothing is given to anyone
    c.count = 1
    table, (lens, count, start, pos, slots) = _extend(c, new, 20)
    with pytest.raises(WencError, match="free pages out of range") as e:
        sync_status()
    assert e.value.status == 1
    assert np.array_equal(table.cpu().numpy(), c.table) and lens.tolist() == c.lens and count.item() == 1
    assert (start == 0).all() and (pos == 0).all() and (slots == -1).all()
    assert isinstance(table, torch.Tensor)


@pytest.mark.parametrize("case", ["new", "len", "table", "rows", "count", "negative"])
def test_extend_reports_what_is_out_of_range(case):
    from transformer_encoder_gb300 import WencError, sync_status
    c = Cache([5, 20, 40], 16, 4, 9, 2)
    new, rows, lens = [3, 2, 9], 20, list(c.lens)
    if case == "new":
        new[1] = -1
    elif case == "len":
        lens[0] = -5
    elif case == "table":
        new[2] = 25
        rows = 40
    elif case == "rows":
        rows = 13
    elif case == "count":
        c.count = len(c.free) + 1
    else:
        c.count = -1
    table, got = _extend(c, new, rows, lens)
    with pytest.raises(WencError, match="out of range"):
        sync_status()
    assert np.array_equal(table.cpu().numpy(), c.table) and got[0].tolist() == lens and got[1].item() == c.count
    assert (got[2] == 0).all() and (got[3] == 0).all() and (got[4] == -1).all()


def test_extend_reports_a_page_below_zero():
    from transformer_encoder_gb300 import WencError, sync_status
    c = Cache([5, 20], 16, 4, 9, 3)
    c.free[c.count - 1] = -4
    table, got = _extend(c, [12, 2], 14)
    with pytest.raises(WencError, match="page number out of range"):
        sync_status()
    assert got[4][:11].min().item() >= 0 and got[4][11].item() == -1 and got[4][12:].min().item() >= 0


@pytest.mark.parametrize("n,past,page,window,sinks,done", [
    (1, 40, 16, 0, 0, 1.0), (1, 40, 16, 10, 1, 0.0), (5, 100, 8, 30, 20, 0.5), (256, 2000, 16, 0, 0, 0.2),
    (700, 300, 1, 50, 4, 0.1), (5000, 400, 16, 60, 4, 0.05), (33, 900, 24, 5000, 0, 0.4), (64, 200, 16, 1, 0, 0.0)])
def test_release(n, past, page, window, sinks, done):
    import torch
    from transformer_encoder_gb300 import kv_release, sync_status
    r = np.random.default_rng(n + past)
    lens = r.integers(0, past + 1, n).tolist()
    fin = r.random(n) < done
    first = -(-sinks // page) if window else 0
    gone = [max(0, m - int(r.integers(0, 3 * page)) - window + 1) // page if window else 0 for m in lens]
    c = Cache(lens, page, -(-past // page) + 1, 3, n, lambda s, e: e < first or e >= gone[s])
    free, count, marks = c.free.copy(), c.count, []
    for s, m in enumerate(lens):
        total, end = -(-m // page), max(0, m - window + 1) // page if window else 0
        give = [e for e in range(total) if (fin[s] and (e < first or e >= gone[s])) or (not fin[s] and max(first, gone[s]) <= e < end)]
        for e in give:
            free[count] = c.table[s, e]
            count += 1
        marks.append(0 if fin[s] else max(end, gone[s]))
    tf = torch.from_numpy(c.free).cuda()
    table = torch.from_numpy(c.table).cuda()
    got = kv_release(_t(lens), table, tf, _t([c.count]), page, finished=torch.from_numpy(fin).cuda() if done else None,
                     window=window or None, sinks=sinks, trimmed=_t(gone) if window else None) if done or window else None
    sync_status()
    assert got[0].tolist() == [0 if f else m for f, m in zip(fin, lens)] and got[1].item() == count
    assert np.array_equal(tf.cpu().numpy(), free) and np.array_equal(table.cpu().numpy(), c.table)
    assert (got[2] is None) == (not window) and (not window or got[2].tolist() == marks)


@pytest.mark.parametrize("case", ["len", "long", "mark", "room", "count"])
def test_release_reports_what_is_out_of_range(case):
    import torch
    from transformer_encoder_gb300 import WencError, kv_release, sync_status
    c = Cache([50, 20, 40], 16, 4, 2, 5)
    lens, gone, count, free = list(c.lens), [0, 0, 0], c.count, c.free
    if case == "len":
        lens[1] = -1
    elif case == "long":
        lens[0] = 65
    elif case == "mark":
        gone[2] = 5
    elif case == "room":
        free = free[:6]
    else:
        count = -1
    tf = torch.from_numpy(free.copy()).cuda()
    got = kv_release(_t(lens), torch.from_numpy(c.table).cuda(), tf, _t([count]), 16,
                     finished=torch.tensor([True, False, True], device="cuda"), window=17, sinks=0, trimmed=_t(gone))
    with pytest.raises(WencError, match="out of range"):
        sync_status()
    assert got[0].tolist() == lens and got[1].item() == count and got[2].tolist() == gone
    assert np.array_equal(tf.cpu().numpy(), free)


def test_no_sequences():
    import torch
    from transformer_encoder_gb300 import kv_extend, kv_release, sync_status
    none, table = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    lens, count, start, pos, slots = kv_extend(none, none, table, _t([4, 5]), _t([2]), 16, 5)
    assert lens.numel() == 0 and count.item() == 2 and start.tolist() == [0] and pos.tolist() == [0] * 5 and slots.tolist() == [-1] * 5
    lens, count, _ = kv_release(none, table, _t([4, 5]), _t([2]), 16, finished=torch.zeros(0, dtype=torch.bool, device="cuda"))
    assert lens.numel() == 0 and count.item() == 2
    sync_status()


def test_what_the_binding_refuses():
    import torch
    from transformer_encoder_gb300 import kv_extend, kv_release
    c = Cache([5, 20], 16, 4, 9, 3)
    table, free = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.free).cuda()
    a = [_t([1, 1]), _t(c.lens), table, free, _t([c.count]), 16, 2]
    for i, x in ((0, a[0].long()), (0, _t([1])), (1, a[1].cpu()), (2, table.long()), (2, table[:1]), (3, free.long()), (4, _t([1, 2])),
                 (5, 0), (6, -1)):
        with pytest.raises(Exception):
            kv_extend(*[x if j == i else y for j, y in enumerate(a)])
    for kw in (dict(lens_out=a[1]), dict(free_count_out=a[4]), dict(positions=_t([0])), dict(slots=_t([0, 0]))):
        with pytest.raises(Exception):
            kv_extend(*a, **kw)
    b = [a[1], table, free, a[4], 16]
    fin = torch.tensor([True, False], device="cuda")
    for kw in (dict(), dict(finished=fin.int()), dict(finished=fin, trimmed=_t([0, 0])), dict(window=5), dict(window=0, trimmed=_t([0, 0])),
               dict(finished=fin, lens_out=a[1]), dict(finished=fin, sinks=-1)):
        with pytest.raises(Exception):
            kv_release(*b, **kw)
