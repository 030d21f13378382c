"""Page bookkeeping on the device against a plain Python reference: every table, count, length and page byte."""

import ctypes
import os
import random
import shutil
import subprocess

import numpy as np
import pytest
import torch

import paged_kv_decode_pda_gb300 as pda
from paged_kv_decode_pda_gb300 import _binding, build
from tests import ops_util as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Both:
    """The reference pool and the device's, moved in step."""

    def __init__(self, NB, rows, cols, bs=16, arrays=((64,), (48,)), seed=0):
        self.ref = O.Pool(NB, rows, cols, bs)
        self.bs = bs
        self.dev = self.ref.tensors(DEV)
        rng = np.random.default_rng(seed)
        self.pages = [rng.integers(0, 256, (NB,) + tuple(s), dtype=np.uint8) for s in arrays]
        self.caches = [torch.from_numpy(p.copy()).to(DEV) for p in self.pages]

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device=DEV).view(-1)

    def step(self, what, *lists, copies=True, status=None):
        getattr(self.ref, what)(*lists)
        fn = getattr(pda, what + "_pages")
        args = [self.i32(x) for x in lists]
        if what in ("fork", "compact"):
            fn(*self.dev, *args, self.bs, self.caches if copies else ())
            if copies:
                for p in self.pages:
                    self.ref.apply_moves(p)
        else:
            fn(*self.dev, *args, self.bs)
        want = (128 if self.ref.refused else 0) if status is None else status
        assert pda.query_device_status() == want, what
        self.same(what)

    def same(self, what=""):
        refs, tables, lens = (x.cpu() for x in self.dev)
        assert refs.tolist() == self.ref.refs, what
        assert lens.tolist() == self.ref.lens, what
        assert tables.tolist() == self.ref.tables, what
        for p, c in zip(self.pages, self.caches):
            assert np.array_equal(c.cpu().numpy(), p), what


def test_a_small_walk():
    b = Both(40, 6, 8)
    b.step("grow", [0, 1], [33, 16])
    b.step("fork", [0, 1], [2, 3])
    b.step("grow", [2, 0, 3], [20, 0, 1])
    b.step("free", [0])
    b.step("grow", [4], [100])
    b.step("compact")
    b.step("free", [1, 2, 3, 4])
    assert b.ref.refs == [0] * 40


@pytest.mark.parametrize("seed,NB,rows,cols,bs,arrays", [
    (0, 60, 10, 12, 16, ((64,),)), (1, 300, 40, 20, 32, ((8, 128, 32), (8, 32, 4))),
    (2, 9000, 300, 70, 16, ((16,), (32,))), (3, 20000, 64, 400, 48, ()), (4, 33, 33, 3, 128, ((20000,),)),
    (5, 5000, 1500, 5, 64, ((160,),) * 3)])
def test_random_walks(seed, NB, rows, cols, bs, arrays):
    rng = random.Random(seed)
    b = Both(NB, rows, cols, bs, arrays, seed)
    for step in range(24):
        used = [r for r in range(rows) if b.ref.lens[r]]
        empty = [r for r in range(rows) if not b.ref.lens[r]]
        what = rng.choice(["grow", "grow", "grow", "fork", "fork", "free", "compact"])
        if what == "grow":
            pick = rng.sample(range(rows), rng.randint(1, rows)) + [-1] * rng.randrange(3)
            most = max(2, int(2.2 * NB * bs / len(pick) / 3))
            b.step("grow", pick, [rng.randrange(min(most, cols * bs)) for _ in pick])
        elif what == "fork" and used and empty:
            kids = rng.sample(empty, rng.randint(1, len(empty)))
            b.step("fork", [rng.choice(used + [-1] if rng.random() < 0.2 else used) for _ in kids], kids)
        elif what == "free" and used:
            b.step("free", rng.sample(used, rng.randint(1, len(used))) + [-1])
        elif what == "compact":
            b.step("compact")


def test_more_requests_than_a_block_of_threads():
    b = Both(5000, 3000, 4, arrays=())
    b.step("grow", list(range(2500)), [1 + i % 40 for i in range(2500)])
    b.step("free", list(range(0, 2500, 3)))
    b.step("fork", list(range(1, 400, 3)) * 3, list(range(2500, 2899)))


def test_refusals_leave_the_state_alone():
    b = Both(4, 5, 4)
    b.step("grow", [0, 0, 9, 1, 2], [20, 5, 1, 70, -1])        # a repeat, no such row, past the row, less than nothing
    assert b.ref.refused == 4 and b.ref.lens == [20, 0, 0, 0, 0]
    b.step("grow", [1, 2, 3], [20, 30, 0])                      # the second finds no page; nothing is needed for the third
    assert b.ref.lens == [20, 20, 0, 0, 0]
    b.step("fork", [0, 1], [2, 3])                              # no page left for a partly filled one
    assert b.ref.refused == 2
    b.step("free", [1, 1, 77, -3])                              # twice: freed once; 77: no such row
    b.step("fork", [0, 0, 0, 2, 4], [1, 1, 0, 3, 4])            # a repeat, a child that holds tokens and is a parent, ...
    b.step("fork", [0], [9])


def test_ids_outside_the_pool_are_flagged_and_skipped():
    b = Both(8, 3, 4)
    b.step("grow", [0], [40])
    b.dev[1][0, 1] = 99
    pda.free_pages(*b.dev, b.i32([0]), 16)
    assert pda.query_device_status() == 64
    assert b.dev[0].tolist() == [0, 1, 0, 0, 0, 0, 0, 0] and b.dev[2].tolist() == [0, 0, 0]


def test_freeing_a_free_page_is_flagged():
    b = Both(8, 2, 4)
    b.step("grow", [0], [20])
    b.dev[0][1] = 0
    pda.free_pages(*b.dev, b.i32([0]), 16)
    assert pda.query_device_status() == 128
    assert b.dev[0].tolist() == [0] * 8


@pytest.mark.parametrize("NB", [40, 9000])
def test_compact_tells_the_new_ids(NB):
    b = Both(NB, 4, 6)
    b.step("grow", [0, 1, 2], [90, 40, 60])
    b.step("free", [0])
    b.dev[0][NB - 1] = 1                      # held outside the table
    b.ref.refs[NB - 1] = 1
    want = list(range(NB))
    b.ref.compact()
    for src, dst in b.ref.moves:
        want[src] = dst
    for p in b.pages:
        b.ref.apply_moves(p)
    ids = torch.full((NB,), -9, dtype=torch.int32, device=DEV)
    pda.compact_pages(*b.dev, 16, b.caches, new_ids=ids)
    assert ids.tolist() == want and want[NB - 1] < NB - 1
    b.same()


def test_copy_pages():
    NB = 50
    rng = np.random.default_rng(0)
    pages = [rng.integers(0, 256, (NB,) + s, dtype=np.uint8) for s in ((16,), (8, 2048), (16400,), (2, 3, 16))]
    caches = [torch.from_numpy(p.copy()).to(DEV) for p in pages]
    src, dst = [3, -1, 7, 3, 9, 60, 2, 5], [40, 41, -2, 42, 9, 43, 99, 0]
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pda.copy_pages(caches, t(src), t(dst))
    assert pda.query_device_status() == 64
    for p, c in zip(pages, caches):
        for s, d in ((3, 40), (3, 42), (5, 0)):
            p[d] = p[s]
        assert np.array_equal(c.cpu().numpy(), p)


def test_more_arrays_than_a_launch_takes():
    b = Both(30, 4, 6, arrays=((32,),) * 131)
    b.step("grow", [0, 1], [40, 50])
    b.step("free", [0])
    b.step("fork", [1], [2])
    b.step("compact")


def test_a_pool_past_2_31_bytes():
    NB = 1 << 16
    cache = torch.zeros(NB, 40000, dtype=torch.uint8, device=DEV)
    assert cache.numel() > 1 << 31
    cache[NB - 1] = 7
    cache[NB - 2, ::3] = 9
    last = cache[NB - 2].clone()
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pda.copy_pages([cache], t([NB - 1, NB - 2]), t([1, NB - 3]))
    assert (cache[1] == 7).all() and torch.equal(cache[NB - 3], last) and (cache[0] == 0).all()


def test_captured_with_a_reserved_workspace():
    b = Both(64, 6, 8)
    b.step("grow", [0, 1], [20, 35])
    parents, kids, rows, add = b.i32([0, 1]), b.i32([2, 3]), b.i32([0, 1, 2, 3]), b.i32([3, 14, 1, 30])
    s = torch.cuda.Stream(priority=-1)   # apart from the streams that other tests draw
    s.wait_stream(torch.cuda.current_stream())
    pda.reserve_pages(64, 6, 4, stream=s)
    s.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        pda.fork_pages(*b.dev, parents, kids, 16, b.caches)
        pda.grow_pages(*b.dev, rows, add, 16)
        pda.free_pages(*b.dev, kids, 16)
        pda.compact_pages(*b.dev, 16, b.caches)
    for _ in range(3):
        gr.replay()
        torch.cuda.synchronize()
        for what, lists in (("fork", ([0, 1], [2, 3])), ("grow", ([0, 1, 2, 3], [3, 14, 1, 30])), ("free", ([2, 3],)),
                            ("compact", ())):
            getattr(b.ref, what)(*lists)
            if what in ("fork", "compact"):
                for p in b.pages:
                    b.ref.apply_moves(p)
        b.same()
    assert pda.query_device_status() == 0


def test_a_capture_that_would_grow_the_workspace_is_refused():
    b = Both(64, 6, 8)
    s = torch.cuda.Stream(priority=-1)   # apart from the streams that other tests draw
    rows = b.i32([0])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        with pytest.raises(pda.PdaError) as e:
            pda.grow_pages(*b.dev, rows, rows, 16)
        assert e.value.status == pda.PDA_ERR_WORKSPACE
        b.dev[2].add_(0)


def test_empty_pools_and_lists():
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    b = Both(5, 2, 3)
    pda.grow_pages(*b.dev, z, z, 16)
    pda.fork_pages(*b.dev, z, z, 16, b.caches)
    pda.free_pages(*b.dev, z, 16)
    pda.copy_pages(b.caches, z, z)
    b.step("compact")
    pda.compact_pages(z, torch.zeros(0, 4, dtype=torch.int32, device=DEV), z, 16)
    b.step("grow", [0, 1], [0, 0])


@pytest.fixture(scope="module")
def threads(tmp_path_factory):
    """tests/page_threads.c beside the loaded library."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    pda.load()
    out = str(tmp_path_factory.mktemp("threads") / "page_threads.so")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run([gcc, "-std=gnu11", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-pthread",
                    "-I", os.path.join(build.ROOT, "include"), os.path.join(here, "page_threads.c"), "-o", out,
                    _binding.LIB_PATH, "-Wl,-rpath," + os.path.dirname(os.path.abspath(_binding.LIB_PATH))], check=True)
    return ctypes.CDLL(out)


def counts_follow_the_table(refs, tables, lens, bs):
    held = torch.zeros(refs.shape[0], dtype=torch.int32)
    for row, n in zip(tables.cpu(), lens.tolist()):
        held.index_add_(0, row[:-(-n // bs)].long(), torch.ones(-(-n // bs), dtype=torch.int32))
    assert torch.equal(held, refs.cpu())


def test_freeing_beside_a_compaction(threads):
    # threads on one stream: a call of one never falls between two kernels of another's
    b = Both(4000, 40, 60, arrays=((32,),))
    pda.grow_pages(*b.dev, b.i32(list(range(40))), b.i32([500 + 7 * r for r in range(40)]), 16)
    rows, add = b.i32(list(range(0, 40, 3)) + list(range(1, 40, 3)) + [-1]), b.i32([400] * 14)
    table, _ = _binding._page_table("", *b.dev, 16)
    array = _binding._PageArray(b.caches[0].data_ptr(), 32)
    pda.reserve_pages(4000, 40, 14)
    torch.cuda.synchronize()
    assert threads.churn_beside_compaction(ctypes.byref(table), ctypes.byref(array), 1, ctypes.c_void_p(rows.data_ptr()),
                                           ctypes.c_void_p(add.data_ptr()), 14, 5000,
                                           ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    assert pda.query_device_status() == 0
    counts_follow_the_table(*b.dev, 16)


class Decoded:
    """Rows of random pages whose K is the first and whose V the last of many arrays, so that their copies take many
    launches; decoded by a thread of its own while a page call runs in another."""

    H, K, NB, ROWS, COLS, ARRAYS = 4, 1, 80, 8, 12, 1300

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.k = O.e4m3(self.NB, self.K, 8, 16, 16, g=g).to(DEV)
        self.v = O.e4m3(self.NB, self.K, 128, 16, g=g).to(DEV)
        self.rest = torch.zeros(self.ARRAYS - 2, self.NB, 16, dtype=torch.uint8, device=DEV)
        self.q = torch.randn(self.ROWS, self.H, 128, generator=g).to(torch.bfloat16).to(DEV)
        i32 = torch.int32
        self.state = (torch.zeros(self.NB, dtype=i32, device=DEV), torch.zeros(self.ROWS, self.COLS, dtype=i32, device=DEV),
                      torch.zeros(self.ROWS, dtype=i32, device=DEV))

    def grow(self, rows, add):
        t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        pda.grow_pages(*self.state, t(rows), t(add), 16)

    def free(self, rows):
        pda.free_pages(*self.state, torch.tensor(rows, dtype=torch.int32, device=DEV), 16)

    def beside(self, threads, parents=None, children=None, loops=60):
        """The outputs [loops, ROWS, H, 128] of decodes beside the call, and of one behind it."""
        table, _ = _binding._page_table("", *self.state, 16)
        bases = [(self.k.data_ptr(), 2048)] + [(x.data_ptr(), 16) for x in self.rest] + [(self.v.data_ptr(), 2048)]
        arrays = (_binding._PageArray * self.ARRAYS)(*bases)
        out = torch.full((loops, self.ROWS, self.H, 128), 77.0, dtype=torch.bfloat16, device=DEV)
        p, c = (None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV) for x in (parents, children))
        pda.reserve(self.ROWS, self.H, self.K, self.COLS, 16)
        pda.reserve_pages(self.NB, self.ROWS, self.ROWS)
        torch.cuda.synchronize()
        ptr = lambda x: ctypes.c_void_p(None if x is None else x.data_ptr())  # noqa: E731
        st = threads.decode_beside_pages(ctypes.byref(table), arrays, self.ARRAYS, ptr(p), ptr(c),
                                         0 if p is None else len(parents), ptr(self.q), self.H, self.K, ptr(out),
                                         ctypes.c_size_t(out[0].nbytes), loops,
                                         ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0 and pda.query_device_status() == 0
        end = pda.decode(self.q, self.k, self.v, self.state[1], self.state[2], 0.1, 0.05, 0.05)
        return out, end


def test_decoding_beside_a_compaction_of_many_arrays(threads):
    for seed in range(12):
        d = Decoded(seed)
        d.grow([0, 1, 2, 3, 4, 5], [160, 150, 170, 90, 150, 111])
        d.free([0, 1])
        out, end = d.beside(threads)
        assert d.state[1][2:6, :6].max() < 36, "nothing was moved"
        assert (out == end).all(), seed


def test_decoding_beside_a_fork(threads):
    # a child's row is empty or whole, never a length with another's pages
    for seed in range(12):
        d = Decoded(seed)
        d.grow([0, 1, 2], [160, 150, 171])
        d.state[1][4:] = torch.randint(40, 80, (4, 12), dtype=torch.int32, device=DEV)   # left from earlier owners
        out, end = d.beside(threads, [0, 1, 2, 2], [4, 5, 6, 7])
        assert torch.equal(d.state[2][4:], d.state[2][[0, 1, 2, 2]])
        assert (out[:, :3] == end[:3]).all() and (out[:, 3] == 0).all(), seed
        for r in range(4, 8):
            for x in out[:, r]:
                assert (x == 0).all() or torch.equal(x, end[r]), (seed, r)


@pytest.mark.parametrize("NB", [60, 9000])
@pytest.mark.parametrize("above", [False, True])
def test_compacting_a_table_that_names_a_free_page(NB, above):
    # the entry stays as it is and is flagged, whether its page lies below or above the held ones' number
    b = Both(NB, 4, 8)
    b.step("grow", [0, 1, 2], [90, 70, 100])
    b.step("free", [0])
    stale = NB - 3 if above else 2               # 0..5 are row 0's old pages; 12 are held
    was = int(b.dev[1][2, 1])
    b.dev[1][2, 1] = stale
    b.dev[0][was] = 0
    b.ref.tables[2][1] = stale
    b.ref.refs[was] = 0
    pda.compact_pages(*b.dev, 16, b.caches)
    assert pda.query_device_status() == 128
    tables = b.dev[1].tolist()
    b.ref.compact()
    b.ref.tables[2][1] = stale
    assert tables == b.ref.tables and b.dev[0].tolist() == b.ref.refs
