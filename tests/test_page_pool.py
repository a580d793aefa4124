"""The host page pool (sequences of pages that grow, fork without a copy, are cut back and released): bookkeeping only,
so every test here runs without a GPU."""
import random
import threading

import pytest

import kv_cache_token_fx_gb300 as fx


@pytest.fixture(scope="module", autouse=True)
def lib():
    from kv_cache_token_fx_gb300 import build
    build.build()
    return fx.load_library()


def test_grow_fork_copy_on_write_release():
    p = fx.PagePool(8, 16, max_seqs=3, max_pages=4)
    a = p.open()
    assert a == 0 and p.append(a, 20) is None and p.free_pages() == 6 and p.length(a) == 20
    b = p.fork(a)                                   # shares both pages
    assert b == 1 and p.free_pages() == 6
    table, length = p.batch([a, b])
    assert table[0].tolist() == table[1].tolist() == [0, 1, -1, -1] and length.tolist() == [20, 20]
    assert p.append(b, 0) is None                   # nothing will be written
    assert p.append(b, 1) == (1, 2)                 # the half-filled page is shared: b gets its own
    assert p.append(b, 1) is None and p.append(a, 3) is None
    table, length = p.batch([b, a])
    assert table[:, :2].tolist() == [[0, 2], [0, 1]] and length.tolist() == [22, 23]
    assert p.release(a) == 1                        # page 0 is still b's
    assert p.release(b) == 2 and p.free_pages() == 8
    assert p.open() == 0


def test_full_pages_are_shared_without_copies():
    p = fx.PagePool(4, 16, max_seqs=2, max_pages=4)
    a = p.open()
    p.append(a, 32)
    b = p.fork(a)
    assert p.append(b, 1) is None and p.append(a, 1) is None
    t, _ = p.batch([a, b])
    assert t[0, :2].tolist() == t[1, :2].tolist() and t[0, 2] != t[1, 2]
    assert p.truncate(b, 20) == 1 and p.length(b) == 20       # its third page; the second stays shared
    own = int(t[1, 2])                                        # the page that b gave back is the next to be given out
    assert p.append(b, 5) == (int(t[0, 1]), own)


def test_errors_change_nothing():
    p = fx.PagePool(3, 16, max_seqs=2, max_pages=3)
    a = p.open()
    p.append(a, 17)
    b = p.fork(a)
    for call in (lambda: p.append(a, 40), lambda: p.append(b, 32), lambda: p.append(a, -1), lambda: p.append(5, 1),
                 lambda: p.fork(a), lambda: p.open(), lambda: p.truncate(a, 18), lambda: p.truncate(a, -1),
                 lambda: p.append(a, (1 << 32) + 1), lambda: p.fork(1 << 32), lambda: p.release((1 << 32) + a),
                 lambda: p.release(2), lambda: p.release(-1), lambda: p.length(9), lambda: p.batch([a, 7])):
        with pytest.raises(fx.FxError):
            call()
        assert p.free_pages() == 1 and p.length(a) == p.length(b) == 17
        assert p.batch([a])[0].tolist() == p.batch([b])[0].tolist() == [[0, 1, -1]]
    assert p.append(b, 1) == (1, 2)                 # the last free page
    with pytest.raises(fx.FxError):
        p.append(a, 16)
    assert p.batch([])[0].shape == (0, 3)
    for sizes in ((0, 16, 1, 1), (1, 0, 1, 1), (1, 16, 0, 1), (1, 16, 1, 0), (1, 1 << 20, 1, 1 << 12)):
        with pytest.raises(fx.FxError):
            fx.PagePool(*sizes)


def test_random_runs_keep_every_sequences_rows():
    """Rows are written through the tables as a caller would (copies included): no sequence ever sees another's."""
    for seed in range(20):
        r = random.Random(seed)
        rows, pages = r.choice([1, 4, 16]), 24
        p = fx.PagePool(pages, rows, max_seqs=6, max_pages=8)
        store, want, tick = [[None] * rows for _ in range(pages)], {}, 0
        for _ in range(300):
            op = r.random()
            live = list(want)
            try:
                if op < 0.15 or not live:
                    want[p.open()] = []
                elif op < 0.55:
                    s, n = r.choice(live), r.randint(0, 2 * rows + 1)
                    pair = p.append(s, n)
                    if pair:
                        store[pair[1]] = list(store[pair[0]])
                    table = p.batch([s])[0][0].tolist()
                    for _ in range(n):
                        at, tick = len(want[s]), tick + 1
                        store[table[at // rows]][at % rows] = tick
                        want[s].append(tick)
                elif op < 0.75:
                    s = r.choice(live)
                    want[p.fork(s)] = list(want[s])
                elif op < 0.9:
                    s = r.choice(live)
                    n = r.randint(0, len(want[s]))
                    p.truncate(s, n)
                    want[s] = want[s][:n]
                else:
                    s = r.choice(live)
                    p.release(s)
                    del want[s]
            except fx.FxError:
                pass
            used = set()
            for s, w in want.items():
                table, length = p.batch([s])
                t = table[0].tolist()
                assert length.tolist() == [len(w)] and t.count(-1) == 8 - -(-len(w) // rows)
                assert [store[t[i // rows]][i % rows] for i in range(len(w))] == w
                used |= {x for x in t if x >= 0}
            assert p.free_pages() == pages - len(used)


def test_threads():
    p = fx.PagePool(64, 16, max_seqs=16, max_pages=4)

    def work():
        for _ in range(200):
            s = p.open()
            p.append(s, 20)
            f = p.fork(s)
            p.append(f, 20)
            p.release(s)
            p.release(f)

    ts = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert p.free_pages() == 64
