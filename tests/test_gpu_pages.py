"""Forking, compacting and copying pages against a step-by-step plan in plain Python (exact)."""
import numpy as np
import pytest
import torch

import kv_cache_block_lowrank_gb300 as hss

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_block_lowrank_gb300 import _build

    _build.build()
    hss.load()


def plan_fork(tables, refs, released, parents, lengths, room, bs):
    """The documented rules, one after another."""
    pages = len(refs)
    ok = lambda p: 0 <= p < pages
    refs = list(refs)
    for p in [p for t in tables for p in t] + list(released):
        if ok(p):
            refs[p] -= 1
    heirs = []
    for i, p in enumerate(parents):
        t = tables[p] if 0 <= p < len(tables) else []
        n = min(max(lengths[i], 0), len(t) * bs)
        r = max(room[i], 0)
        kept = list(t[:-(-n // bs)])
        heirs.append((kept, -(-(n + r) // bs), r > 0 and n % bs != 0 and ok(kept[-1])))
        for p in kept:
            if ok(p):
                refs[p] += 1
    owners = {}
    for i, (kept, _, writes) in enumerate(heirs):
        if writes:
            owners.setdefault(kept[-1], []).append(i)
    own = {p: (w[0] if refs[p] == len(w) else None) for p, w in owners.items()}
    for p, w in owners.items():
        refs[p] -= len(w) - (own[p] is not None)
    free = [p for p in range(pages) if refs[p] == 0]
    new, copies, missing = [], [], 0
    for i, (kept, n, writes) in enumerate(heirs):
        t = list(kept)
        copy = t.pop() if writes and own[kept[-1]] != i else None
        first = True
        while len(t) < n:
            p = free.pop(0) if free else -1
            missing += p < 0
            if p >= 0:
                refs[p] = 1
            if copy is not None and first:
                copies.append((copy, p))
            first = False
            t.append(p)
        new.append(t)
    return new, refs, copies, missing


def run_fork(tables, refs, released, parents, lengths, room, bs, table_room=None, total=None,
             fill=0xEE):
    flat = [p for t in tables for p in t]
    offs = np.cumsum([0] + [len(t) for t in tables])
    need = sum(-(-(min(max(n, 0), len(tables[p]) * bs if 0 <= p < len(tables) else 0)
                   + max(r, 0)) // bs) for p, n, r in zip(parents, lengths, room))
    table_room = need + 5 if table_room is None else table_room
    new = len(parents)
    t = lambda x: torch.tensor(x, **I32)
    guard = 123456
    out = {k: torch.full((n + 2,), guard, **I32) for k, n in
           dict(table=table_room, offs=new + 1, refs=len(refs), src=new, dst=new,
                counts=4).items()}
    size = hss.hss_fork_pages_workspace_bytes(new, len(refs))
    work = torch.full((size + 8,), fill, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, **I32)
    hss.hss_fork_pages(t(flat), t(offs), len(tables), len(flat), t(refs), len(refs),
                       t(released) if len(released) else None, len(released), t(parents),
                       t(lengths), t(room), new, bs, table_room, out["table"], out["offs"],
                       out["refs"], out["src"], out["dst"], out["counts"], work, size, status)
    torch.cuda.synchronize()
    assert (work[size:] == fill).all()
    got = {}
    for k, v in out.items():
        v = v.tolist()
        assert v[-2:] == [guard] * 2, k
        got[k] = v[:-2]
    return got, status.item(), table_room


def check_fork(args, got, table_room):
    new, refs, copies, missing = plan_fork(*args)
    flat = [p for t in new for p in t]
    pad = lambda x, n: x + [-1] * (n - len(x))
    assert got["offs"] == np.cumsum([0] + [len(t) for t in new]).tolist()
    assert got["table"] == pad(flat, table_room)
    assert got["refs"] == refs
    assert got["src"] == pad([a for a, _ in copies], len(new))
    assert got["dst"] == pad([b for _, b in copies], len(new))
    assert got["counts"] == [len(flat), len(copies), sum(r != 0 for r in refs), missing]


def random_state(g, seqs, most, pages, shared, extra):
    """Tables with common prefixes, counts with holders besides the tables."""
    ids = g.permutation(pages).tolist()
    prefix = [ids.pop() for _ in range(shared)]
    tables = []
    for _ in range(seqs):
        t = prefix[:int(g.integers(0, shared + 1))]
        t += [ids.pop() for _ in range(int(g.integers(0, most + 1)))]
        tables.append(t)
    refs = np.bincount(np.array([p for t in tables for p in t], dtype=int), minlength=pages)
    held = g.integers(0, pages, extra).tolist()
    for p in held:
        refs[p] += 1
    return tables, refs.tolist(), held


@pytest.mark.parametrize("seqs,new,most,pages,bs", [
    (1, 1, 3, 16, 16), (4, 16, 5, 120, 16), (7, 3, 9, 100, 48), (64, 64, 20, 4000, 16),
    (300, 700, 12, 9000, 32), (3, 2500, 40, 20000, 16), (5, 40, 2000, 70000, 16)])
def test_fork_plans(seqs, new, most, pages, bs):
    g = np.random.default_rng(seqs * new + pages)
    tables, refs, held = random_state(g, seqs, most, pages, 3, 4)
    parents = g.integers(-1, seqs, new).tolist()
    lengths = [int(g.integers(-2, len(tables[p]) * bs + 3)) if g.random() < 0.7
               else len(tables[p]) * bs - int(g.integers(0, 3)) for p in parents]
    room = [int(x) for x in g.choice([0, 0, 1, 2, bs, 3 * bs + 1, -4], new)]
    args = (tables, refs, held[:2] + [-1], parents, lengths, room, bs)
    got, status, table_room = run_fork(*args)
    assert status == (hss.HSS_ERR_OUT_OF_RANGE if got["counts"][3] else 0)
    hss.hss_read_device_error()
    check_fork(args, got, table_room)


def test_fork_by_hand():
    """Two sequences on a common page; one goes on, one forks in three and writes, one is new."""
    tables, refs = [[5, 2], [5, 7]], [0, 0, 1, 0, 0, 2, 0, 1]
    got, status, _ = run_fork(tables, refs, [], [0, 1, 1, -1], [20, 30, 20, 9], [0, 4, 1, 17], 16,
                              table_room=9)
    # 0 keeps 5, 2 and writes nothing; 1 and 2 both write into 7: 1 keeps it, 2 gets a copy in
    # page 1 (1 needs page 0 for its third entry first); 3 begins with nothing: pages 3 and 4
    assert got["table"] == [5, 2, 5, 7, 0, 5, 1, 3, 4] and status == 0
    assert got["offs"] == [0, 2, 5, 7, 9]
    assert got["src"] == [7, -1, -1, -1] and got["dst"] == [1, -1, -1, -1]
    assert got["refs"] == [1, 1, 1, 1, 1, 3, 0, 1] and got["counts"] == [9, 1, 7, 0]


def test_a_reader_keeps_the_page_from_its_writers():
    """A page that one heir keeps whole and two write into the middle of: both get copies."""
    tables, refs = [[0]], [1, 0, 0, 0]
    args = (tables, refs, [], [0, 0, 0], [16, 10, 4], [0, 1, 1], 16)
    got, status, room = run_fork(*args)
    check_fork(args, got, room)
    assert status == 0 and got["src"][:2] == [0, 0] and got["dst"][:2] == [1, 2]
    # so does somebody besides the tables
    args = (tables, [2, 0, 0, 0], [], [0], [10], [1], 16)
    got, status, room = run_fork(*args)
    check_fork(args, got, room)
    assert got["dst"][0] == 1 and got["refs"] == [1, 1, 0, 0]


def test_fork_errors():
    read = hss.hss_read_device_error
    # too few pages: the last entries are missing, the copy's page first if it comes first
    args = ([[0], [1]], [1, 1, 0], [], [0, 0, 1], [5, 5, 16], [40, 1, 1], 16)
    got, status, room = run_fork(*args)
    check_fork(args, got, room)
    assert status == hss.HSS_ERR_OUT_OF_RANGE == read() and got["counts"][3] == 3
    assert got["dst"][0] == -1 and got["src"][0] == 0
    # parents and ids that do not exist
    args = ([[0, 9, -3]], [1, 0, 0, 0], [77], [0, 5, -4], [40, 16, 16], [0, 3, 1], 16)
    got, status, room = run_fork(*args)
    check_fork(args, got, room)
    assert status == hss.HSS_ERR_OUT_OF_RANGE == read()
    # a table that is too small: nothing past its end is touched (run_fork looks), sizes are right
    got, status, _ = run_fork([[0, 1]], [1, 1, 0, 0], [], [0, 0], [32, 32], [16, 16], 16,
                              table_room=3)
    assert status == hss.HSS_ERR_INVALID_ARGUMENT == read()
    assert got["counts"][0] == 6 and got["offs"] == [0, 3, 6]
    # counts that are too small
    _, status, _ = run_fork([[0, 1]], [1, 0, 0], [], [0], [32], [0], 16)
    assert status == hss.HSS_ERR_INVALID_ARGUMENT == read()
    # nothing at all
    got, status, _ = run_fork([], [0, 2], [], [], [], [], 16, table_room=2)
    assert status == 0 and got["table"] == [-1, -1] and got["counts"] == [0, 0, 1, 0]


@pytest.mark.parametrize("held,writers,pages", [(2, 2, 4), (3, 2, 40), (2, 5, 5000), (40, 41, 9000)])
def test_fork_counts_too_small(held, writers, pages):
    """Counts below what the tables give up are an error, and every id is still one of the pool's,
    whatever the workspace held (here words that read as ids far behind it)."""
    tables = [[1]] * held + [[3]]
    parents = [0] * writers + [held]
    for count in range(-1, held):
        refs = [0] * pages
        refs[1], refs[3] = count, 1
        room = [1] * writers + [16 * pages]        # all that is free is handed out
        got, status, _ = run_fork(tables, refs, [], parents, [5] * writers + [16], room, 16,
                                  fill=0x7F)
        assert status in (hss.HSS_ERR_INVALID_ARGUMENT, hss.HSS_ERR_OUT_OF_RANGE)
        assert all(-1 <= p < pages for k in ("table", "src", "dst") for p in got[k])
    hss.hss_read_device_error()


def test_fork_without_room_for_the_table():
    """Copies into entries that the new table has no room for have nowhere to go."""
    got, status, _ = run_fork([[1, 2]], [0, 1, 1, 0, 0, 0], [], [0, 0, 0], [20] * 3, [1] * 3, 16,
                              table_room=2)
    assert status == hss.HSS_ERR_INVALID_ARGUMENT
    assert got["counts"][0] == 6 and got["offs"] == [0, 2, 4, 6]
    assert got["dst"] == [-1] * 3
    hss.hss_read_device_error()


def run_compact(table, refs, move_room):
    t = lambda x: torch.tensor(x, **I32)
    guard = 123456
    out = {k: torch.full((n + 2,), guard, **I32) for k, n in
           dict(table=len(table), refs=len(refs), src=move_room, dst=move_room,
                counts=4).items()}
    size = hss.hss_compact_pages_workspace_bytes(len(refs))
    work = torch.full((size + 8,), 0xEE, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, **I32)
    hss.hss_compact_pages(t(table), len(table), t(refs), len(refs), move_room, out["table"],
                          out["refs"], out["src"], out["dst"], out["counts"], work, size, status)
    torch.cuda.synchronize()
    assert (work[size:] == 0xEE).all()
    got = {}
    for k, v in out.items():
        v = v.tolist()
        assert v[-2:] == [guard] * 2, k
        got[k] = v[:-2]
    return got, status.item()


@pytest.mark.parametrize("pages,share,move_room", [
    (1, 1.0, 3), (2, 0.5, 2), (33, 0.4, 40), (1000, 0.5, 7), (1000, 0.9, 1000), (5000, 0.0, 3),
    (5000, 1.0, 3), (70000, 0.3, 70000), (70001, 0.7, 100), (4097, 0.5, 0)])
def test_compact_plans(pages, share, move_room):
    g = np.random.default_rng(pages + move_room)
    refs = (g.random(pages) < share) * g.integers(1, 4, pages)
    used = np.flatnonzero(refs)
    table = np.concatenate([g.permutation(np.repeat(used, refs[used])), [-1]]).astype(int)
    got, status = run_compact(table.tolist(), refs.tolist(), move_room)
    assert status == 0
    n = len(used)
    holes = [p for p in range(n) if refs[p] == 0]
    tops = used[used >= n][::-1].tolist()
    moves = list(zip(tops, holes))[:move_room]
    want_refs, goes = refs.copy(), np.arange(pages)
    for src, dst in moves:
        want_refs[dst], want_refs[src], goes[src] = refs[src], 0, dst
    pad = lambda x: x + [-1] * (move_room - len(x))
    assert got["src"] == pad([a for a, _ in moves]) and got["dst"] == pad([b for _, b in moves])
    assert got["refs"] == want_refs.tolist()
    assert got["table"] == goes[table[:-1]].tolist() + [-1]
    last = max(np.flatnonzero(want_refs).tolist() + [-1]) + 1
    assert got["counts"] == [len(moves), n, last, len(tops) - len(moves)]


def test_compact_errors():
    got, status = run_compact([3, 99, -2, 1], [0, 1, 0, 1], 4)
    assert status == hss.HSS_ERR_OUT_OF_RANGE == hss.hss_read_device_error()
    assert got["table"] == [0, 99, -2, 1] and got["refs"] == [1, 1, 0, 0]
    got, status = run_compact([2], [-1, 0, 1], 2)
    assert status == hss.HSS_ERR_INVALID_ARGUMENT == hss.hss_read_device_error()
    assert got["refs"] == [-1, 1, 0] and got["table"] == [1]


@pytest.mark.parametrize("page,pages,layers,copies,two", [
    (16, 8, 1, 3, False), (18432, 20, 3, 9, True), (16400, 33, 2, 16, True),
    (48, 5000, 1, 2400, False), (1 << 20, 6, 2, 3, True)])
def test_copies(page, pages, layers, copies, two):
    g = torch.Generator(device=DEV).manual_seed(page + pages)
    pools = [torch.randint(0, 256, (layers, pages, page), generator=g, device=DEV,
                           dtype=torch.uint8) for _ in range(2 if two else 1)]
    ids = torch.randperm(pages, generator=g, device=DEV).int()
    src, dst = ids[:copies].clone(), ids[copies:2 * copies].clone()
    src[copies // 2], dst[0] = -1, (-1 if copies > 4 else dst[0])
    if copies > 2:
        src[2] = src[1]  # one page copied twice
    for count in (None, copies - 1, 0, copies + 9, -3):
        number = None if count is None else torch.tensor([count], **I32)
        n = copies if count is None else max(0, min(count, copies))
        want = [p.clone() for p in pools]
        got = [p.clone() for p in pools]
        there = (src[:n] >= 0) & (dst[:n] >= 0)
        for w in want:
            w[:, dst[:n][there].long()] = w[:, src[:n][there].long()]
        hss.hss_copy_pages(src, dst, number, copies, got[0], got[1] if two else None, page, pages,
                           layers)
        torch.cuda.synchronize()
        assert hss.hss_read_device_error() == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_copies_of_pages_that_do_not_exist_and_past_32_bits():
    pages, page, layers = 40, 1 << 25, 4   # 5 GB
    pool = torch.zeros(layers, pages, page, device=DEV, dtype=torch.uint8)
    g = torch.Generator(device=DEV).manual_seed(1)
    pool[:, 39] = torch.randint(0, 256, (layers, page), generator=g, device=DEV,
                                dtype=torch.uint8)
    src = torch.tensor([39, 40, 1, 1 << 30], **I32)
    dst = torch.tensor([2, 3, 40, 4], **I32)
    status = torch.zeros(1, **I32)
    hss.hss_copy_pages(src, dst, None, 4, pool, None, page, pages, layers, status)
    torch.cuda.synchronize()
    assert status.item() == hss.HSS_ERR_OUT_OF_RANGE == hss.hss_read_device_error()
    assert torch.equal(pool[:, 2], pool[:, 39])
    assert not pool[:, 3:39].any() and not pool[:, :2].any()
