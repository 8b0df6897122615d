"""kva_extend_page_tables against its definition, request by request (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kva():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_kv_cache_mla_gb300 import kva

    return kva


def expected(table, lens, new, free, taken, page, num_pages):
    """(table, slots, taken, flags) by walking the tokens."""
    table, slots, flags = table.clone(), [], 0
    taken = min(taken, len(free))
    for b, (n, length) in enumerate(zip(new, lens)):
        for pos in range(length, length + n):
            idx, row = pos // page, pos % page
            if idx >= table.shape[1]:
                slots.append(-1)
                flags = 1
                continue
            if row == 0:
                got = free[taken] if taken < len(free) else -1
                taken = min(taken + 1, len(free))
                table[b, idx] = got if 0 <= got < num_pages else -1
            got = int(table[b, idx])
            ok = 0 <= got < num_pages
            slots.append(got * page + row if ok else -1)
            flags |= 0 if ok else 1
    return table, torch.tensor(slots, dtype=torch.int64), taken, flags


class Batch:
    def __init__(self, seed, new, lens, page, *, width=None, spare=5, taken=3, short=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens, self.page = list(new), list(lens), page
        have = [-(-p // page) for p in self.lens]
        need = [-(-(p + n) // page) for n, p in zip(self.new, self.lens)]
        self.num_pages = sum(need) + spare + taken
        ids = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        self.table = torch.full((len(self.new), max(need + [1]) + 1 if width is None else width), -1,
                                dtype=torch.int32)
        at = 0
        for b, n in enumerate(have):
            n = min(n, self.table.shape[1])
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.free = ids[at:] if not short else ids[at:at + taken + short]
        self.taken = taken
        self.offsets = torch.tensor([0] + list(torch.tensor(self.new).cumsum(0)), dtype=torch.int32)

    def run(self, kva, in_place=False, slots=True, stream=None):
        want = expected(self.table, self.lens, self.new, self.free.tolist(), self.taken, self.page,
                        self.num_pages)
        T = sum(self.new)
        d = dict(table=self.table.cuda(), lens=torch.tensor(self.lens, dtype=torch.int64).to(
            torch.int32).cuda(), off=self.offsets.cuda(), free=self.free.cuda(),
            taken=torch.tensor([self.taken], dtype=torch.int32).cuda())
        out = d["taken"] if in_place else torch.full((1,), 77, dtype=torch.int32, device="cuda")
        slot_map = torch.full((T,), 99, dtype=torch.int64, device="cuda") if slots else None
        fl = torch.zeros(1, dtype=torch.int32, device="cuda")
        kva.kva_extend_page_tables(d["table"], d["lens"], d["off"], d["free"], d["taken"], out,
                                   self.page, self.num_pages, slot_map=slot_map, err_flags=fl,
                                   tot_seq_len=T)
        torch.cuda.synchronize()
        assert torch.equal(d["table"].cpu(), want[0])
        if slots:
            assert torch.equal(slot_map.cpu(), want[1])
        assert int(out) == want[2] and int(fl) == want[3]
        return want


@pytest.mark.parametrize("page", [1, 3, 16, 64, 100])
@pytest.mark.parametrize("in_place", [False, True])
def test_mixed_requests(kva, page, in_place):
    Batch(1, [1, 0, 5, 1, 200, 1, 64, 0, 1], [0, 7, 62, 63, 10, 64, 64, 0, 99], page).run(
        kva, in_place)


def test_one_token(kva):
    for length in (0, 1, 15, 16, 17):
        Batch(2, [1], [length], 16).run(kva, True)


def test_many_tokens_over_the_cluster(kva):
    Batch(3, [5000, 1, 0, 9000, 3000], [100, 200, 300, 0, 17], 16).run(kva, True)


@pytest.mark.parametrize("n", [1023, 1024, 1025, 3000, 8192])
def test_many_requests(kva, n):
    Batch(4, [(i * 7) % 3 for i in range(n)], [(i * 13) % 40 for i in range(n)], 8).run(kva, True)


def test_no_slot_map(kva):
    Batch(5, [3, 40], [5, 0], 16).run(kva, slots=False)


@pytest.mark.parametrize("short", [1, 2, 4])
def test_the_list_ends(kva, short):
    want = Batch(6, [40, 1, 40, 1], [5, 16, 0, 7], 16, short=short).run(kva, True)
    assert want[3] == 1


def test_more_taken_than_there_are(kva):
    b = Batch(7, [40, 1], [5, 16], 16)
    b.taken = len(b.free) + 9
    b.run(kva, True)


def test_no_free_pages(kva):
    b = Batch(8, [3, 1], [5, 16], 16)
    b.free, b.taken = b.free[:0], 0
    b.run(kva)


def test_invalid_ids(kva):
    b = Batch(9, [40, 1, 2], [5, 20, 31], 16)
    b.free[4] = b.num_pages + 3
    b.table[1, 1] = -1
    assert b.run(kva)[3] == 1


@pytest.mark.parametrize("width", [1, 2, 3])
def test_past_the_table(kva, width):
    """What lies past the table's width takes no page."""
    assert Batch(10, [40, 1, 9], [5, 70, 30], 16, width=width).run(kva)[3] == 1


@pytest.mark.parametrize("length", [0x7FFFFFFF, 0x80000000, 0xFFFFFFFF])
def test_the_longest_lengths(kva, length):
    b = Batch(11, [2, 3], [5, 6], 16)
    b.lens = [length, 6]
    want = (b.table.clone(), None, None, 1)
    lens = torch.tensor([length - (1 << 32) if length >> 31 else length, 6], dtype=torch.int32)
    table, fl = b.table.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(5, dtype=torch.int64, device="cuda")
    taken = torch.tensor([3], dtype=torch.int32, device="cuda")
    kva.kva_extend_page_tables(table, lens.cuda(), b.offsets.cuda(), b.free.cuda(), taken, taken,
                               16, b.num_pages, slot_map=slots, err_flags=fl)
    torch.cuda.synchronize()
    page = int(b.table[1, 0])
    assert slots.tolist() == [-1, -1] + [page * 16 + r for r in (6, 7, 8)]
    assert int(fl) == 1 and int(taken) == 3 and torch.equal(table.cpu(), want[0])


@pytest.mark.parametrize("offsets", [[1, 2, 3], [0, 1, 2], [0, 4, 3], [0, 1, 9]])
def test_malformed_offsets(kva, offsets):
    b = Batch(12, [1, 2], [16, 16], 16)
    table, fl = b.table.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.full((3,), 99, dtype=torch.int64, device="cuda")
    taken = torch.tensor([3], dtype=torch.int32, device="cuda")
    kva.kva_extend_page_tables(table, torch.tensor(b.lens, dtype=torch.int32).cuda(),
                               torch.tensor(offsets, dtype=torch.int32).cuda(), b.free.cuda(),
                               taken, taken, 16, b.num_pages, slot_map=slots, err_flags=fl)
    torch.cuda.synchronize()
    assert int(fl) == 4 and int(taken) == 3
    assert torch.equal(table.cpu(), b.table) and bool((slots == 99).all())


def test_captured_steps(kva):
    """A graph of one decode step, replayed: lengths grow on the device, pages
    are taken as they are needed."""
    b = Batch(13, [1, 1, 1], [14, 15, 0], 16, spare=20)
    table, free = b.table.cuda(), b.free.cuda()
    lens = torch.tensor(b.lens, dtype=torch.int32).cuda()
    off = b.offsets.cuda()
    taken = torch.tensor([b.taken], dtype=torch.int32).cuda()
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    fl = torch.zeros(1, dtype=torch.int32, device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    wide = torch.nn.functional.pad(table, (0, 4), value=-1).contiguous()
    b.table = torch.nn.functional.pad(b.table, (0, 4), value=-1)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        kva.kva_extend_page_tables(wide, lens, off, free, taken, taken, 16, b.num_pages,
                                   slot_map=slots, err_flags=fl, stream=s)
        lens.add_(1)
    for _ in range(40):
        b.table, want, b.taken, flags = expected(b.table, b.lens, b.new, b.free.tolist(), b.taken,
                                                 16, b.num_pages)
        b.lens = [n + 1 for n in b.lens]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(slots.cpu(), want) and torch.equal(wide.cpu(), b.table)
        assert int(taken) == b.taken and int(fl) == flags == 0
