"""kv_pages_grow and kv_pages_trim on the GPU against lists and loops: whole numbers, equal."""

import numpy as np
import pytest

import oracle.step as ref
import weight_streaming_linear_amd as wsl
from gpu_common import say

pytestmark = pytest.mark.gpu


def _state(g, n, per, page, n_pages, fill=0.5, pad=0):
    """A KVPages with sequences of random lengths and its reference."""
    import torch
    lens, table, numbers = [], np.full((n, per), -7, np.int32), list(g.permutation(n_pages))
    for b in range(n):
        length = int(g.integers(0, per * page + 1) * fill)
        length = min(length, len(numbers) * page)
        held = -(-length // page)
        table[b, :held] = [numbers.pop() for _ in range(held)]
        lens.append(length)
    n_free = len(numbers)
    free = np.array(numbers + [-9] * (n_pages - n_free), np.int32)
    wide = torch.full((n, per + pad), -7, dtype=torch.int32, device="cuda")
    wide[:, :per] = torch.from_numpy(table).cuda()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pages = wsl.KVPages(wide[:, :per], dev(lens), torch.from_numpy(free).cuda(), dev([n_free]), page)
    return pages, ref.Pages(table, lens, free, n_free, page)


def _same(pages, want):
    assert pages.lens.tolist() == want.lens
    assert pages.n_free.tolist() == [want.n_free]
    assert pages.free.tolist() == want.free
    assert pages.table.tolist() == want.table


def _grow(pages, want, new, n_tokens, uniform=False, st=None):
    import torch
    starts = torch.full((pages.n_seq + 1,), -5, dtype=torch.int32, device="cuda")
    arg = new[0] if uniform else torch.tensor(new, dtype=torch.int32, device="cuda")
    slots, positions = wsl.kv_pages_grow(pages, arg, n_tokens=n_tokens, starts=starts, status=st)
    w = want.grow(new, n_tokens)
    assert starts.tolist() == w[2]
    assert positions.tolist() == w[1]
    assert slots.tolist() == w[0]
    _same(pages, want)


def _trim(pages, want, to, st=None):
    import torch
    wsl.kv_pages_trim(pages, torch.tensor(to, dtype=torch.int32, device="cuda"), status=st)
    want.trim(to)
    _same(pages, want)


@pytest.mark.parametrize("n,per,page,new", [(1, 4, 16, 1), (1, 1, 1, 1), (5, 40, 1, 3), (7, 9, 7, 5), (64, 12, 16, 5),
                                            (300, 6, 24, 8), (1023, 3, 20, 1), (1024, 3, 16, 5), (1025, 3, 16, 2),
                                            (3, 600, 16, 3000), (2, 70, 128, 4097), (2500, 2, 5, 3)])
def test_steps_against_lists(n, per, page, new):
    """Steps of one launch and of two, uniform and ragged, drafts taken back, sequences ended and begun again."""
    import torch
    say(f"pages n={n} per={per} page={page} new={new}")
    g = np.random.default_rng([2026, 21, n, new])
    pages, want = _state(g, n, per, page, max(1, int(0.8 * n * per)), pad=3)
    for step in range(4):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        want.status = 0
        uniform = step % 2 == 0
        grow = [min(new, per * page)] * n if uniform else g.integers(0, min(new, per * page) + 1, n).tolist()
        _grow(pages, want, grow, sum(grow) + (step == 3) * 5, uniform, st)
        assert st.item() == want.status
        to = [int(x) for x in np.maximum(np.array(want.lens) - g.integers(0, new + 1, n), 0)]
        for b in g.integers(0, n, 1 + n // 10):
            to[b] = int(g.choice([0, 1 << 30, want.lens[b]]))
        _trim(pages, want, to)


def test_growing_again_takes_the_same_pages():
    g = np.random.default_rng([2026, 22])
    pages, want = _state(g, 50, 30, 16, 2000)
    before, free = pages.lens.clone(), pages.free.clone()
    first, _ = wsl.kv_pages_grow(pages, 40)
    table = pages.table.clone()
    wsl.kv_pages_trim(pages, before)
    assert pages.free.equal(free) and pages.lens.equal(before)
    again, _ = wsl.kv_pages_grow(pages, 40)
    assert again.equal(first) and pages.table.equal(table)


@pytest.mark.parametrize("n", [6, 1500])
def test_too_few_pages(n):
    """From the first sequence that lacks one on, only those that need none go on."""
    import torch
    page, per = 8, 4
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    lens = [8, 3, 16, 8, 7, 8] + [5] * (n - 6)
    table = np.arange(n * per, dtype=np.int32).reshape(n, per)
    free = [7, 9, 11] + [0] * (n * per - 3)
    for n_free in (0, 1, 2, 3):
        pages = wsl.KVPages(torch.from_numpy(table).cuda(), dev(lens), dev(free), dev([n_free]), page)
        want = ref.Pages(table, lens, free, n_free, page)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        new = [1, 2, 9, 1, 1, 1] + [3] * (n - 6)
        _grow(pages, want, new, sum(new), st=st)
        assert st.item() == want.status == wsl.WSL_STATUS_PAGES


@pytest.mark.parametrize("n", [6, 1500])
def test_bad_numbers_are_left_out_and_reported(n):
    """Lengths and growths out of range, tokens past the room, page numbers that name no page, a stack
    that cannot be: nothing is read or written out of bounds, the rest goes on."""
    import torch
    g = np.random.default_rng([2026, 23, n])
    page, per = 8, 4
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")

    def fresh(lens, n_free, free=None):
        table = g.permutation(n * per * 2)[:n * per].astype(np.int32).reshape(n, per)
        free = list(range(n * per * 2)) if free is None else free
        pages = wsl.KVPages(torch.from_numpy(table).cuda(), dev(lens), dev(free), dev([n_free]), page)
        return pages, ref.Pages(table, lens, free, n_free, page), torch.zeros(1, dtype=torch.int32, device="cuda")

    base = [3] * n
    for at, length, grow in [(2, -1, 1), (2, -2 ** 31, 1), (0, 33, 1), (2, 2 ** 31 - 1, 1), (2, 32, 1), (2, 30, 3),
                             (2, 3, -1), (2, 3, -2 ** 31), (2, 3, 2 ** 31 - 1), (5, 0, 33)]:
        lens, new = list(base), [5] * n
        lens[at], new[at] = length, grow
        pages, want, st = fresh(lens, n * per)
        _grow(pages, want, new, 5 * (n + 7), st=st)
        assert st.item() == want.status != 0
    pages, want, st = fresh(base, n * per)
    _grow(pages, want, [5] * n, 17, st=st)                              # room for three of them
    assert st.item() == want.status == wsl.WSL_STATUS_INDEX
    for n_free in (-1, -2 ** 31, 2 * n * per + 1, 2 ** 31 - 1):
        pages, want, st = fresh(base, n_free)
        _grow(pages, want, [5] * n, 5 * n, st=st)
        assert st.item() == want.status and st.item() & wsl.WSL_STATUS_INDEX
    pages, want, st = fresh(base, n * per, [2 * n * per, -1, 2 ** 31 - 1, -2 ** 31, 5] * (2 * n * per // 5 + 1))
    _grow(pages, want, [9] * n, 9 * n, st=st)
    assert st.item() == want.status == wsl.WSL_STATUS_INDEX
    for lens, to in [([-1] + base[1:], [0] * n), ([33] + base[1:], [0] * n), (base, [-1] + [0] * (n - 1)),
                     (base, [-2 ** 31] + [2 ** 31 - 1] * (n - 1))]:
        pages, want, st = fresh(lens, n * per)
        _trim(pages, want, to, st)
        assert st.item() == want.status == wsl.WSL_STATUS_INDEX
    pages, want, st = fresh(base, 2 * n * per - 3)                      # no room to give pages back
    _trim(pages, want, [0] * n, st)
    assert st.item() == want.status == wsl.WSL_STATUS_INDEX


def test_no_sequences_and_no_tokens():
    import torch
    pages = wsl.KVPages(torch.empty(0, 3, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"),
                        torch.arange(4, dtype=torch.int32, device="cuda"), torch.tensor([4], dtype=torch.int32, device="cuda"), 16)
    starts = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    slots, positions = wsl.kv_pages_grow(pages, 1, n_tokens=5, starts=starts)
    assert slots.tolist() == positions.tolist() == [-1] * 5 and starts.tolist() == [0]
    assert wsl.kv_pages_grow(pages, 1)[0].numel() == 0
    wsl.kv_pages_trim(pages, torch.empty(0, dtype=torch.int32, device="cuda"))
    pages, want = _state(np.random.default_rng(5), 9, 3, 4, 30)
    _grow(pages, want, [0] * 9, 0)


def test_a_long_row():
    """Positions and slots at the far end of 2^31 - 1 tokens."""
    import torch
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    page, lens = 1 << 20, [2 ** 31 - 10, 2 ** 31 - 3, 5]
    table = (np.arange(3 * 2048).reshape(3, 2048) + 2 ** 31 - 7000).astype(np.int32)
    pages = wsl.KVPages(torch.from_numpy(table).cuda(), dev(lens), torch.arange(9, dtype=torch.int32, device="cuda"), dev([9]), page)
    pages.desc.n_pages = 2 ** 31 - 1            # only the table's numbers are this far
    slots, positions = wsl.kv_pages_grow(pages, 4)
    at = [lens[0] + i for i in range(4)]
    assert positions.tolist()[:4] == at and slots.tolist()[:4] == [int(table[0, 2047]) * page + p % page for p in at]
    assert slots.tolist()[4:8] == [-1] * 4 and pages.lens.tolist() == [lens[0] + 4, lens[1], 9]


def test_a_captured_step_moves_on_by_itself():
    """grow and trim in one graph: every replay takes the next tokens, the drafts fall again."""
    import torch
    g = np.random.default_rng([2026, 24])
    pages, want = _state(g, 40, 20, 8, 700, fill=0.2)
    saved = [t.clone() for t in (pages.table, pages.lens, pages.free, pages.n_free)]
    to = torch.empty(40, dtype=torch.int32, device="cuda")
    slots, positions = (torch.empty(200, dtype=torch.int64, device="cuda") for _ in range(2))

    def step():
        wsl.kv_pages_grow(pages, 5, slots=slots, positions=positions)
        torch.sub(pages.lens, 3, out=to)
        wsl.kv_pages_trim(pages, to)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    for t, x in zip((pages.table, pages.lens, pages.free, pages.n_free), saved):
        t.copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        graph.replay()
        w = want.grow([5] * 40, 200)
        want.trim([n - 3 for n in want.lens])
        assert slots.tolist() == w[0] and positions.tolist() == w[1]
        _same(pages, want)
