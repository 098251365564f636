"""The paged key/value cache: tables from request lengths, append, attention of
new tokens, and a serving loop of the three, against the oracle."""
import ctypes

import numpy as np
import pytest

from oracle import window_oracle as wo
from trainable_block_sparse_compressed_b200 import infllmv2 as host_api

from _helpers import f64
from test_window_attn import FAKE, check


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------
def i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32).cuda()


def run_tables(api, kv, q, free, table, page, n_tokens, n_pages):
    import torch
    n, width = len(kv), len(table[0])
    p = api.make_paged_params(n, width, n_pages, page, n_tokens=n_tokens)
    t = i32(table)
    free_t = i32(free) if free else torch.empty(0, dtype=torch.int32, device="cuda")
    out = dict(cu=i32([-9] * (n + 1)), lens=i32([-9] * n), left=i32([-9]),
               slots=torch.full((n_tokens,), -9, dtype=torch.int32, device="cuda"),
               pos=torch.full((n_tokens,), -9, dtype=torch.int32, device="cuda"))
    api.paged_tables(p, i32(kv), i32(q), free_t, i32([len(free)]), t, out["cu"], out["lens"],
                     out["slots"], out["pos"], out["left"])
    torch.cuda.synchronize()
    return (t.cpu().tolist(), out["cu"].tolist(), out["lens"].tolist(), out["slots"].tolist(),
            out["pos"].tolist(), out["left"].item())


def make_tables(seed, n, max_kv, max_q, page):
    r = np.random.default_rng(seed)
    kv = r.integers(0, max_kv + 1, n).tolist()
    q = r.integers(0, max_q + 1, n).tolist()
    have = [-(-k // page) for k in kv]
    width = max(1, max(-(-(k + x) // page) for k, x in zip(kv, q)))
    pages = r.permutation(sum(have) + n * (max_q // page + 2)).tolist()
    table, at = [], 0
    for h in have:
        table.append(pages[at:at + h] + [-1] * (width - h))
        at += h
    return kv, q, pages[at:], table, len(pages)


@pytest.mark.gpu
@pytest.mark.parametrize("n,max_kv,max_q,page,pad", [
    (1, 0, 1, 64, 0), (1, 300, 1, 16, 2), (5, 130, 0, 64, 3), (33, 1000, 1, 64, 0),
    (100, 700, 90, 16, 11), (1024, 500, 40, 32, 1), (1025, 2000, 3, 128, 0), (3000, 100, 9, 16, 5),
    (8192, 64, 2, 64, 0), (7, 5000, 3000, 128, 1),
])
def test_paged_tables(cuda_lib, n, max_kv, max_q, page, pad):
    kv, q, free, table, n_pages = make_tables(n + page, n, max_kv, max_q, page)
    n_tokens = sum(q) + pad
    got = run_tables(cuda_lib, kv, q, free, table, page, n_tokens, n_pages)
    *ref, fine = wo.paged_tables(kv, q, free, table, page, n_tokens)
    assert fine and got == tuple(ref)
    assert cuda_lib.get_status() == 0


@pytest.mark.gpu
def test_paged_tables_out_of_pages(cuda_lib):
    api = cuda_lib
    args = ([5, 8, 0], [20, 10, 40], [3, 4], [[0, -1, -1], [1, -1, -1], [-1, -1, -1]], 16, 71)
    kv, q, free, table, page, n = args
    got = run_tables(api, kv, q, free, table, page, n, 5)
    # the pages go to the requests in order: one to request 0, one to request 1
    *ref, fine = wo.paged_tables(kv, q, free, table, page, n)
    assert not fine and got == tuple(ref)
    assert api.get_status() == api.STATUS_NO_PAGE
    assert api.get_status() == 0


@pytest.mark.gpu
def test_paged_tables_with_an_empty_free_list(cuda_lib):
    """No page left and none needed, then one needed: an empty list is a list."""
    api = cuda_lib
    args = ([5, 30], [2, 2], [], [[0, -1], [2, 1]], 16, 4)
    *ref, fine = wo.paged_tables(*args)
    assert fine and run_tables(api, *args, 3) == tuple(ref)
    assert api.get_status() == 0
    args = ([16, 30], [2, 2], [], [[0, -1], [2, 1]], 16, 4)
    *ref, fine = wo.paged_tables(*args)
    assert not fine and run_tables(api, *args, 3) == tuple(ref)
    assert api.get_status() == api.STATUS_NO_PAGE


@pytest.mark.gpu
def test_paged_tables_too_long_and_negative(cuda_lib):
    """A sequence that outgrows its table row, more tokens than rows, and
    lengths below zero: nothing is written outside, the status says so."""
    api = cuda_lib
    kv, q, free, table = [20, -5, 3], [30, -2, 4], [9, 8, 7, 6], [[0, 1], [-1, -1], [2, -1]]
    got = run_tables(api, kv, q, free, table, 16, 32, 10)
    *ref, fine = wo.paged_tables(kv, q, free, table, 16, 32)
    assert not fine and got == tuple(ref)
    assert api.get_status() == api.STATUS_SEQ_FULL


@pytest.mark.gpu
def test_paged_tables_take_no_page_for_a_column_that_the_table_lacks(cuda_lib):
    """Two of four requests outgrow their rows of three columns: the free list
    loses the pages that were entered and no others, and the requests behind
    them get theirs."""
    api, page = cuda_lib, 16
    kv, q = [40, 0, 60, 10], [30, 100, 1, 20]
    table = [[0, 1, 2], [-1, -1, -1], [3, 4, 5], [6, -1, -1]]
    free = [7, 8, 9, 10, 11]
    got = run_tables(api, kv, q, free, table, page, 151, 12)
    # request 1 takes three pages, request 3 one
    assert got[0] == [[0, 1, 2], [11, 10, 9], [3, 4, 5], [6, 8, -1]] and got[5] == 1
    *ref, fine = wo.paged_tables(kv, q, free, table, page, 151)
    assert not fine and got == tuple(ref)
    assert api.get_status() == api.STATUS_SEQ_FULL
    # a request already past its row takes none either
    got = run_tables(api, [70], [5], [1, 2], [[0, 3, 4]], page, 5, 5)
    assert got == ([[0, 3, 4]], [0, 5], [75], [-1] * 5, [70, 71, 72, 73, 74], 2)
    assert api.get_status() == api.STATUS_SEQ_FULL


@pytest.mark.gpu
def test_paged_tables_replayed_after_a_shortage_keep_reporting_it(cuda_lib):
    """Lengths in place, the list short by a page in the first step: the steps
    after it find the entry at -1 and say so, until a page is entered."""
    import torch
    api, page = cuda_lib, 16
    p = api.make_paged_params(2, 4, 6, page, n_tokens=4)
    lens, q, table = i32([15, 31]), i32([2, 2]), i32([[0, -1, -1, -1], [1, 2, -1, -1]])
    free, count = i32([3]), i32([1])
    cu, slots, pos = i32([0] * 3), i32([0] * 4), i32([0] * 4)

    def step():
        api.paged_tables(p, lens, q, free, count, table, cu, lens, slots, pos, count)
        return api.get_status(), slots.tolist()

    assert step() == (api.STATUS_NO_PAGE, [15, 48, 47, -1])
    assert step() == (api.STATUS_NO_PAGE, [49, 50, -1, -1])
    table[1, 2] = 4
    assert step() == (0, [51, 52, 67, 68])
    table[1, 2] = 6      # not a page of the pool
    assert step() == (api.STATUS_NO_PAGE, [53, 54, -1, -1])
    torch.cuda.synchronize()
    assert count.item() == 0 and lens.tolist() == [23, 39]


@pytest.mark.gpu
def test_paged_tables_nonsense_lengths_stay_inside(cuda_lib):
    """Lengths whose sums pass 32 bits: ascending offsets, every slot and entry
    inside, the status set."""
    api = cuda_lib
    n, big = 40, (1 << 31) - 1
    kv, q = [0] * n, [big] * n
    kv[5] = big
    table, cu, lens, slots, pos, left = run_tables(api, kv, q, [3, 1], [[-1, -1]] * n, 16, 100, 4)
    assert cu == sorted(cu) and cu[0] == 0 and cu[-1] == big and left == 0
    assert table[0] == [1, 3] and all(r == [-1, -1] for r in table[1:])
    assert slots[:32] == [16 + i for i in range(16)] + [48 + i for i in range(16)]
    assert slots[32:] == [-1] * 68 and pos == list(range(100))
    assert lens[0] == 1 << 28    # a length is cut there
    assert api.get_status() == api.STATUS_NO_PAGE | api.STATUS_SEQ_FULL


@pytest.mark.gpu
def test_paged_tables_replayed_in_place(cuda_lib):
    """seqlens over kv_lens and the free count in place: a captured step
    replayed 70 times equals 70 steps of the oracle."""
    import torch
    api = cuda_lib
    n, page, steps = 9, 16, 70
    kv, q = [0, 1, 15, 16, 17, 100, 31, 32, 33], [1, 2, 1, 1, 0, 1, 3, 1, 1]
    width = -(-(max(kv) + 3 * steps) // page)
    have = [-(-k // page) for k in kv]
    perm = np.random.default_rng(0).permutation(sum(have) + 200).tolist()
    table, at = [], 0
    for h in have:
        table.append(perm[at:at + h] + [-1] * (width - h))
        at += h
    free = perm[at:]
    p = api.make_paged_params(n, width, len(perm), page, n_tokens=sum(q))
    lens, ql, fr, count, t = i32(kv), i32(q), i32(free), i32([len(free)]), i32(table)
    cu, slots, pos = i32([0] * (n + 1)), i32([0] * sum(q)), i32([0] * sum(q))
    call = lambda: api.paged_tables(p, lens, ql, fr, count, t, cu, lens, slots, pos, count)  # noqa: E731
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            call()
    for _ in range(steps):
        graph.replay()
        table, rcu, kv, rs, rp, left, fine = wo.paged_tables(kv, q, free, table, page, sum(q))
        free = free[:left]
    torch.cuda.synchronize()
    assert fine and t.tolist() == table and lens.tolist() == kv and count.item() == left
    assert slots.tolist() == rs and pos.tolist() == rp and cu.tolist() == rcu
    assert api.get_status() == 0


REFUSED_LAUNCH = """
import torch
from trainable_block_sparse_compressed_b200 import infllmv2 as api
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
p = api.make_paged_params(1, 2, 4, 16, n_tokens=3)
args = [i32(0), i32(3), i32(0, 1, 2, 3), i32(4), i32(-1, -1).view(1, 2), i32(0, 0), i32(0),
        i32(0, 0, 0), i32(0, 0, 0), i32(0)]
K = torch.zeros(4, 16, 1, 128, dtype=torch.bfloat16, device="cuda")
rows = torch.ones(3, 1, 128, dtype=torch.bfloat16, device="cuda")
slots = i32(0, 1, 2)
torch.cuda.synchronize()
side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
codes = []
with torch.cuda.stream(side):
    graph.capture_begin()
    try:
        side.synchronize()          # not allowed in a capture, which it ends
    except RuntimeError:
        pass
    try:
        api.paged_tables(p, *args)
    except api.InfLLMV2Error as e:
        codes.append(e.code)
    try:
        graph.capture_end()
    except RuntimeError:
        pass
api.paged_append(p, slots, rows, rows, K, K.clone())
torch.cuda.synchronize()
assert codes == [api.ERR_CUDA] and float(K.sum()) == 3 * 128
print("fine")
"""


@pytest.mark.gpu
def test_a_refused_launch_fails_its_own_call_alone(cuda_lib):
    """In a process of its own: a capture that was broken off refuses the
    tables' launch; the call after it is not told of that."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", REFUSED_LAUNCH], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout[-1000:] + r.stderr[-2000:]


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("n,Hkv,page,Hq", [(1, 1, 16, 1), (3, 2, 64, 32), (17, 3, 128, 3),
                                           (1000, 8, 32, 16), (4099, 2, 16, 4)])
def test_paged_append(cuda_lib, n, Hkv, page, Hq):
    import torch
    g = torch.Generator().manual_seed(n)
    n_pages = -(-n // page) + 2
    qkv = torch.randn(n, Hq + 2 * Hkv, 128, generator=g).to(torch.bfloat16).cuda()
    K = torch.randn(n_pages, page, Hkv, 128, generator=g).to(torch.bfloat16).cuda()
    V = K.flip(0).contiguous()
    slots = torch.randperm(n_pages * page, generator=g)[:n].to(torch.int32)
    slots[n // 3] = -1                      # skipped
    if n > 2:
        slots[n // 2] = n_pages * page      # outside the pool: skipped
    rK, rV = K.clone().flatten(0, 1), V.clone().flatten(0, 1)
    ok = (slots >= 0) & (slots < n_pages * page)
    rK[slots[ok].long().cuda()] = qkv[ok.cuda(), Hq:Hq + Hkv]
    rV[slots[ok].long().cuda()] = qkv[ok.cuda(), Hq + Hkv:]
    p = cuda_lib.make_paged_params(1, 1, n_pages, page, n_tokens=n, Hq=Hkv, Hkv=Hkv)
    cuda_lib.paged_append(p, slots.cuda(), qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], K, V)
    torch.cuda.synchronize()
    assert torch.equal(K.flatten(0, 1), rK) and torch.equal(V.flatten(0, 1), rV)
    # densely packed rows give the same
    K2, V2 = K.clone(), V.clone()
    cuda_lib.paged_append(p, slots.cuda(), qkv[:, Hq:Hq + Hkv].contiguous(),
                          qkv[:, Hq + Hkv:].contiguous(), K2, V2)
    torch.cuda.synchronize()
    assert torch.equal(K, K2) and torch.equal(V, V2)


@pytest.mark.gpu
@pytest.mark.parametrize("n,Hkv,page", [(1, 1, 16), (3, 2, 64), (17, 3, 128), (1000, 8, 32), (4099, 2, 16)])
@pytest.mark.parametrize("form", ["dense", "K dense", "V dense", "strided"])
def test_paged_append_writes_untouched_pools(cuda_lib, n, Hkv, page, form):
    """Pools that no call has written before: every slot's row arrives, densely
    packed or strided, and nothing else changes."""
    import torch
    g = torch.Generator().manual_seed(n)
    n_pages = -(-n // page) + 2
    kv = torch.randn(n, 2 * Hkv + 1, 128, generator=g).to(torch.bfloat16).cuda()
    k, v = kv[:, :Hkv], kv[:, Hkv + 1:]
    if form in ("dense", "K dense"):
        k = k.contiguous()
    if form in ("dense", "V dense"):
        v = v.contiguous()
    K = torch.full((n_pages, page, Hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    V = torch.full_like(K, 9.0)
    slots = torch.randperm(n_pages * page, generator=g)[:n].cuda()
    want = [x.flatten(0, 1).clone() for x in (K, V)]
    want[0][slots], want[1][slots] = k, v
    p = cuda_lib.make_paged_params(1, 1, n_pages, page, n_tokens=n, Hq=Hkv, Hkv=Hkv)
    cuda_lib.paged_append(p, slots.to(torch.int32), k, v, K, V)
    torch.cuda.synchronize()
    assert torch.equal(K.flatten(0, 1), want[0]) and torch.equal(V.flatten(0, 1), want[1])


# ---------------------------------------------------------------------------
# attention over the cache
# ---------------------------------------------------------------------------
class Batch:
    """Sequences of (keys, new tokens) in shuffled pages; what lies behind a
    sequence's last token, in unused pages and in unused table entries is NaN
    or nonsense."""

    def __init__(self, lens, Hq, Hkv, page, seed, pad=0, fused=False):
        import torch
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hq, self.Hkv, self.page = lens, Hq, Hkv, page
        pages = [-(-k // page) for k, _ in lens]
        self.width = max(1, max(pages)) + 1
        self.n_pages = sum(pages) + 2
        perm = torch.randperm(self.n_pages, generator=g).tolist()
        nan = float("nan")
        K = torch.full((self.n_pages, page, Hkv, 128), nan).to(torch.bfloat16)
        V = K.clone()
        self.k, self.v, self.table, at = [], [], [], 0
        for (n, _), w in zip(lens, pages):
            mine = perm[at:at + w]
            at += w
            k = torch.randn(n, Hkv, 128, generator=g).to(torch.bfloat16)
            v = torch.randn(n, Hkv, 128, generator=g).to(torch.bfloat16)
            for c, pg in enumerate(mine):
                m = min(page, n - c * page)
                K[pg, :m], V[pg, :m] = k[c * page:c * page + m], v[c * page:c * page + m]
            self.table.append(mine + [1 << 30] * (self.width - w))
            self.k.append(k)
            self.v.append(v)
        self.cu = np.concatenate([[0], np.cumsum([q for _, q in lens])]).tolist()
        self.rows = self.cu[-1] + pad
        extra = 2 * Hkv if fused else 0
        qkv = torch.randn(self.rows, Hq + extra, 128, generator=g).to(torch.bfloat16).cuda()
        self.Q = qkv[:, :Hq]
        self.K, self.V = K.cuda(), V.cuda()
        self.table_t, self.cu_t, self.len_t = i32(self.table), i32(self.cu), i32([n for n, _ in lens])

    def params(self, api, window=0, n_sink=0, scale=0.0):
        return api.make_paged_params(len(self.lens), self.width, self.n_pages, self.page,
                                     n_tokens=self.rows, Hq=self.Hq, Hkv=self.Hkv, window=window,
                                     n_sink=n_sink, scale=scale)

    def out(self):
        import torch
        return (torch.full((self.rows, self.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda"),
                torch.full((self.rows, self.Hq), 7.0, device="cuda"))

    def run(self, api, window=0, n_sink=0, scale=0.0):
        p = self.params(api, window, n_sink, scale)
        O, lse = self.out()
        ws = api.alloc_paged_workspace(p)
        ws.fill_(0xff)
        api.paged_attn(p, self.Q, self.K, self.V, self.table_t, self.cu_t, self.len_t, O, lse, ws)
        assert api.get_status() == 0
        return O, lse

    def check(self, O, lse, window=0, n_sink=0, scale=0.0, sample=None):
        o, ls, q = f64(O), f64(lse), f64(self.Q)
        for i, (n, m) in enumerate(self.lens):
            rows = np.arange(self.cu[i], self.cu[i] + m)
            if sample is not None and m > sample:
                rows = rows[np.unique(np.linspace(0, m - 1, sample).astype(int))]
            pos = n - m + rows - self.cu[i]
            ref = wo.attention(q[rows], f64(self.k[i]), f64(self.v[i]), pos, window, n_sink, scale)
            check(o[rows], ls[rows], ref, n)
        assert (o[self.cu[-1]:] == 7).all() and (ls[self.cu[-1]:] == 7).all()


PAGED = [
    # lens (keys, new), Hq, Hkv, page, window, n_sink, pad
    ([(1, 1)], 1, 1, 16, 0, 0, 0),
    ([(1, 1), (2, 1), (127, 1), (128, 1), (129, 1)], 32, 2, 64, 0, 0, 2),
    ([(1000, 1), (700, 1), (33, 1), (5, 1)], 32, 2, 64, 0, 0, 0),
    ([(300, 1), (65, 3), (40, 40), (511, 8)], 16, 4, 16, 0, 0, 1),
    ([(260, 130), (129, 129), (64, 64)], 8, 8, 32, 0, 0, 0),        # heads of their own
    ([(513, 257), (700, 20)], 16, 1, 128, 0, 0, 3),
    ([(900, 300), (50, 50), (640, 1)], 8, 4, 64, 100, 0, 0),
    ([(900, 300), (50, 50), (640, 1)], 32, 2, 16, 100, 4, 5),
    ([(2000, 1), (1500, 2), (90, 1)], 4, 2, 16, 130, 64, 0),
    ([(2000, 700)], 32, 2, 64, 1, 0, 0),
    ([(1200, 1200)], 4, 1, 64, 333, 150, 0),
    ([(0, 0), (5, 0), (77, 77), (0, 0), (10, 1), (0, 0)], 16, 2, 16, 0, 0, 4),   # idle sequences
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hq,Hkv,page,window,n_sink,pad", PAGED)
def test_paged_attn_all_elements(cuda_lib, lens, Hq, Hkv, page, window, n_sink, pad):
    b = Batch(lens, Hq, Hkv, page, seed=len(lens) + page, pad=pad, fused=Hq % 3 == 2)
    O, lse = b.run(cuda_lib, window, n_sink)
    b.check(O, lse, window, n_sink)


@pytest.mark.gpu
def test_paged_attn_more_sequences_than_threads(cuda_lib):
    r = np.random.default_rng(1)
    lens = [(int(n), int(min(n, q))) for n, q in zip(r.integers(0, 60, 900), r.integers(0, 4, 900))]
    b = Batch(lens, 4, 2, 16, seed=1, pad=1)
    b.check(*b.run(cuda_lib))


@pytest.mark.gpu
@pytest.mark.parametrize("window,n_sink", [(0, 0), (4096, 64)])
def test_paged_attn_long_sequences_split(cuda_lib, window, n_sink):
    """Few rows over long caches: the keys are split over the SMs and joined."""
    b = Batch([(40000, 1), (131, 1), (9000, 5), (20011, 1)], 32, 2, 64, seed=2)
    b.check(*b.run(cuda_lib, window, n_sink), window, n_sink)


@pytest.mark.gpu
@pytest.mark.parametrize("window,n_sink,Hq,Hkv", [(100, 5, 32, 2), (256, 0, 8, 2), (7, 64, 4, 4)])
def test_paged_attn_chunks_under_short_windows(cuda_lib, window, n_sink, Hq, Hkv):
    b = Batch([(3000, 900), (700, 333), (20, 20), (5000, 1), (64, 0)], Hq, Hkv, 16, seed=4, pad=3)
    b.check(*b.run(cuda_lib, window, n_sink), window, n_sink, sample=150)


@pytest.mark.gpu
def test_paged_attn_sinks_without_a_window(cuda_lib):
    """Every earlier key is visible anyway: the sinks change no bit."""
    import torch
    b = Batch([(900, 300), (640, 1), (77, 77)], 16, 4, 32, seed=13, pad=1)
    want = b.run(cuda_lib, 0, 0)
    for n_sink in (1, 130, 5000):
        got = b.run(cuda_lib, 0, n_sink)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    b.check(*want)


@pytest.mark.gpu
def test_paged_attn_long_chunk(cuda_lib):
    b = Batch([(9000, 2500), (4000, 1), (3000, 777)], 32, 2, 64, seed=3, pad=7, fused=True)
    b.check(*b.run(cuda_lib), sample=40)


@pytest.mark.gpu
def test_paged_attn_equals_window_attn(cuda_lib):
    """A contiguous cache is a pool of pages: the chunk's rows are the whole
    sequence's, within the roundings of two orders of summation."""
    import torch
    from test_window_attn import make, run
    T, q, window, n_sink = 2048, 600, 500, 10
    Q, K, V = make(1, T, 16, 2, seed=11)
    O, lse = run(cuda_lib, Q, K, V, window, n_sink)
    p = cuda_lib.make_paged_params(1, T // 64, T // 64, 64, n_tokens=q, Hq=16, Hkv=2, window=window,
                                   n_sink=n_sink)
    Oc = torch.empty(q, 16, 128, dtype=torch.bfloat16, device="cuda")
    lc = torch.empty(q, 16, device="cuda")
    ws = cuda_lib.alloc_paged_workspace(p)
    cuda_lib.paged_attn(p, Q[0, T - q:], K.view(T // 64, 64, 2, 128), V.view(T // 64, 64, 2, 128),
                        i32([list(range(T // 64))]), i32([0, q]), i32([T]), Oc, lc, ws)
    torch.cuda.synchronize()
    assert (lc - lse[0, :, T - q:].T).abs().max() < 1e-4
    assert (Oc.float() - O[0, T - q:].float()).abs().max() < 2e-2


@pytest.mark.gpu
def test_paged_attn_pages_behind_the_window_may_be_gone(cuda_lib):
    """Pages without a visible key are not read: their entries may be -1."""
    api, window, n_sink, page = cuda_lib, 200, 20, 16
    b = Batch([(1500, 3), (700, 100)], 16, 2, page, seed=4)
    for i, (n, m) in enumerate(b.lens):
        first = n - m - window + 1
        for c in range(len(b.table[i])):
            if c * page >= n_sink and (c + 1) * page <= first:
                b.table[i][c] = -1
    b.table_t = i32(b.table)
    b.check(*b.run(api, window, n_sink), window, n_sink)


@pytest.mark.gpu
def test_paged_attn_rows_without_a_key(cuda_lib):
    """More new tokens than keys: rows at positions below zero see nothing."""
    api = cuda_lib
    b = Batch([(40, 40), (3, 3)], 8, 2, 16, seed=5)
    b.len_t = i32([30, 0])
    O, lse = b.run(api)
    o, ls = f64(O), f64(lse)
    assert (o[:10] == 0).all() and np.isneginf(ls[:10]).all()
    assert (o[40:] == 0).all() and np.isneginf(ls[40:]).all()
    ref = wo.attention(f64(b.Q)[10:40], f64(b.k[0])[:30], f64(b.v[0])[:30], np.arange(30), 0, 0)
    check(o[10:40], ls[10:40], ref, 30)


@pytest.mark.gpu
def test_paged_attn_bad_pages_and_lengths_are_reported(cuda_lib):
    """An id outside the pool, a length past the table and offsets past the
    rows: no access outside, the other sequences as they should be."""
    import torch
    api = cuda_lib
    b = Batch([(300, 2), (200, 1)], 8, 2, 16, seed=6)
    b.table[0][3] = -1
    b.table_t = i32(b.table)
    p, (O, lse) = b.params(api), b.out()
    ws = api.alloc_paged_workspace(p)
    api.paged_attn(p, b.Q, b.K, b.V, b.table_t, b.cu_t, b.len_t, O, lse, ws)
    assert api.get_status() == api.STATUS_BAD_PAGE
    rows = slice(b.cu[1], b.cu[2])
    ref = wo.attention(f64(b.Q)[rows], f64(b.k[1]), f64(b.v[1]), [199], 0, 0)
    check(f64(O)[rows], f64(lse)[rows], ref, 200)
    api.paged_attn(p, b.Q, b.K, b.V, b.table_t, i32([0, 2, 9000]), i32([300, 1 << 30]), O, lse, ws)
    torch.cuda.synchronize()
    api.get_status()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1, -2, -3, "n_pages", (1 << 31) - 1, -(1 << 31)])
@pytest.mark.parametrize("page,window,n_sink", [(16, 0, 0), (64, 150, 20), (128, 0, 0)])
def test_paged_attn_needed_page_outside_the_pool_reads_as_zeros(cuda_lib, bad, page, window, n_sink):
    """Whatever the id: the status is set, and the sequence's rows are those over
    zeros in the page's place (which sees keys 128 .. 128 + page - 1)."""
    api = cuda_lib
    b = Batch([(300, 2), (200, 1), (290, 40)], 8, 2, page, seed=page)
    for i in (0, 2):
        b.table[i][128 // page] = b.n_pages if bad == "n_pages" else bad
        b.k[i][128:128 + page] = 0
        b.v[i][128:128 + page] = 0
    b.table_t = i32(b.table)
    p, (O, lse) = b.params(api, window, n_sink), b.out()
    ws = api.alloc_paged_workspace(p)
    for _ in range(2):
        api.paged_attn(p, b.Q, b.K, b.V, b.table_t, b.cu_t, b.len_t, O, lse, ws)
        assert api.get_status() == api.STATUS_BAD_PAGE
        b.check(O, lse, window, n_sink)


@pytest.mark.gpu
def test_paged_attn_rows_past_n_tokens_are_cut(cuda_lib):
    """Offsets that pass n_tokens: the rows there are keep their positions."""
    api = cuda_lib
    b = Batch([(90, 1), (200, 60)], 16, 2, 16, seed=9)
    b.rows = 21
    b.Q = b.Q[:21]
    O, lse = b.run(api)
    ref = wo.attention(f64(b.Q)[1:], f64(b.k[1]), f64(b.v[1]), np.arange(140, 160), 0, 0)
    check(f64(O)[1:], f64(lse)[1:], ref, 200)
    ref = wo.attention(f64(b.Q)[:1], f64(b.k[0]), f64(b.v[0]), [89], 0, 0)
    check(f64(O)[:1], f64(lse)[:1], ref, 90)


@pytest.mark.gpu
@pytest.mark.parametrize("past,window,n_sink", [(1, 0, 0), (6, 0, 0), (6, 20, 3), (30, 0, 0), (200, 9, 0),
                                                (1 << 29, 0, 0)])
def test_paged_attn_tokens_past_the_table_leave_the_others_their_positions(cuda_lib, past, window,
                                                                           n_sink):
    """A sequence whose new tokens outgrow its table row: rows that have a place
    stand where they stand, the others get O = 0 and lse = -inf."""
    api, page = cuda_lib, 16
    b = Batch([(64, 30), (40, 3), (64, 1), (100, 100)], 8, 2, page, seed=12, pad=2)
    b.width, b.table = 4, [r[:4] for r in b.table]      # room for 64 keys
    b.table_t = i32(b.table)
    b.len_t = i32([64 + past, 40, 64, 100])
    b.k[3], b.v[3] = b.k[3][:64], b.v[3][:64]
    O, lse = b.run(api, window, n_sink)
    o, ls, q = f64(O), f64(lse), f64(b.Q)
    pos = [np.arange(64 + past - 30, 64 + past), np.arange(37, 40), [63], np.arange(100)]
    for i, t in enumerate(pos):
        t, rows = np.asarray(t), np.arange(b.cu[i], b.cu[i + 1])
        has = t < 64
        ref = wo.attention(q[rows[has]], f64(b.k[i]), f64(b.v[i]), t[has], window, n_sink)
        check(o[rows[has]], ls[rows[has]], ref, 64)
        assert (o[rows[~has]] == 0).all() and np.isneginf(ls[rows[~has]]).all()
    assert (o[b.cu[-1]:] == 7).all() and (ls[b.cu[-1]:] == 7).all()


@pytest.mark.gpu
def test_paged_attn_replayed_with_other_lengths_and_two_workspaces(cuda_lib):
    """One captured call serves changing lengths; two calls in flight on two
    streams, a workspace each, give what they give alone."""
    import torch
    api = cuda_lib
    lens = [(700, 1), (5000, 4), (300, 200)]
    b = Batch(lens, 32, 2, 64, seed=7, pad=3)
    p, (O, lse) = b.params(api), b.out()
    ws = api.alloc_paged_workspace(p)
    lt, ct = i32([1, 4, 200]), i32([0, 1, 5, 205])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        api.paged_attn(p, b.Q, b.K, b.V, b.table_t, ct, lt, O, lse, ws)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            api.paged_attn(p, b.Q, b.K, b.V, b.table_t, ct, lt, O, lse, ws)
    lt.copy_(b.len_t)
    graph.replay()
    torch.cuda.synchronize()
    assert api.get_status() == 0
    b.check(O, lse)
    b2 = Batch([(9000, 1), (100, 30)], 32, 2, 16, seed=8)
    want = b2.run(api)
    p2, out2, ws2 = b2.params(api), b2.out(), api.alloc_paged_workspace(b2.params(api))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        api.paged_attn(p, b.Q, b.K, b.V, b.table_t, ct, lt, O, lse, ws, stream=s1)
        api.paged_attn(p2, b2.Q, b2.K, b2.V, b2.table_t, b2.cu_t, b2.len_t, *out2, ws2, stream=s2)
    torch.cuda.synchronize()
    b.check(O, lse)
    assert torch.equal(out2[0], want[0]) and torch.equal(out2[1], want[1])


# ---------------------------------------------------------------------------
# the three together
# ---------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("window,n_sink,page", [(0, 0, 64), (48, 4, 16)])
def test_serving_loop(cuda_lib, window, n_sink, page):
    """Ragged prompts prefilled in chunks, then decoded, all lengths and pages
    on the GPU: tables -> append -> attention, against the oracle over the
    whole sequences."""
    import torch
    api = cuda_lib
    Hq, Hkv, prompts, chunk, steps = 16, 2, [150, 37, 1, 90], 64, 6
    n, total = len(prompts), [x + steps for x in prompts]
    g = torch.Generator().manual_seed(3)
    qkv = [torch.randn(t, Hq + 2 * Hkv, 128, generator=g).to(torch.bfloat16) for t in total]
    width = -(-max(total) // page)
    n_pages = sum(-(-t // page) for t in total)
    K = torch.full((n_pages, page, Hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    V = K.clone()
    lens, count = i32([0] * n), i32([n_pages])
    free = torch.randperm(n_pages, generator=g).to(torch.int32).cuda()
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    rows = n * chunk
    p = api.make_paged_params(n, width, n_pages, page, n_tokens=rows, Hq=Hq, Hkv=Hkv, window=window,
                              n_sink=n_sink)
    ws = api.alloc_paged_workspace(p)
    cu, slots, pos = i32([0] * (n + 1)), i32([0] * rows), i32([0] * rows)
    x = torch.zeros(rows, Hq + 2 * Hkv, 128, dtype=torch.bfloat16, device="cuda")
    O = torch.zeros(rows, Hq, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(rows, Hq, device="cuda")
    done, got = [0] * n, [[] for _ in range(n)]
    while min(t - d for t, d in zip(total, done)) > 0 or any(d < t for t, d in zip(total, done)):
        q = [min(chunk, pr - d) if d < pr else min(1, t - d) for pr, t, d in zip(prompts, total, done)]
        at = np.concatenate([[0], np.cumsum(q)]).tolist()
        for i in range(n):
            x[at[i]:at[i + 1]] = qkv[i][done[i]:done[i] + q[i]].cuda()
        api.paged_tables(p, lens, i32(q), free, count, table, cu, lens, slots, pos, count)
        api.paged_append(p, slots, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], K, V)
        api.paged_attn(p, x[:, :Hq], K, V, table, cu, lens, O, lse, ws)
        assert api.get_status() == 0
        for i in range(n):
            got[i].append((f64(O[at[i]:at[i + 1]]), f64(lse[at[i]:at[i + 1]])))
            done[i] += q[i]
    assert count.item() == 0 and lens.tolist() == total
    for i in range(n):
        a = f64(qkv[i])
        ref = wo.attention(a[:, :Hq], a[:, Hq:Hq + Hkv], a[:, Hq + Hkv:], np.arange(total[i]),
                           window, n_sink)
        check(np.concatenate([o for o, _ in got[i]]), np.concatenate([l for _, l in got[i]]), ref,
              total[i])


@pytest.mark.gpu
@pytest.mark.parametrize("window,n_sink,page", [(0, 0, 64), (20, 3, 16)])
def test_decode_step_captured_and_replayed(cuda_lib, window, n_sink, page):
    """Tables, append and attention of a decode step as one graph, lengths and
    the free count in place: 70 replays with new rows, every row against the
    oracle over the whole sequences."""
    import torch
    api = cuda_lib
    Hq, Hkv, steps, start = 8, 2, 70, [0, 5, 63, 16, 40]
    n, width = len(start), -(-(max(start) + steps) // page)
    g = torch.Generator().manual_seed(17)
    pages = [-(-x // page) for x in start]
    n_pages = sum(-(-(x + steps) // page) for x in start)
    perm = torch.randperm(n_pages, generator=g).tolist()
    table, at = [], 0
    for h in pages:
        table.append(perm[at:at + h] + [-1] * (width - h))
        at += h
    free = perm[at:]
    old = [torch.randn(x, 2 * Hkv, 128, generator=g).to(torch.bfloat16) for x in start]
    new = torch.randn(steps, n, Hq + 2 * Hkv, 128, generator=g).to(torch.bfloat16)
    K = torch.full((n_pages, page, Hkv, 128), float("nan"), dtype=torch.bfloat16)
    V = K.clone()
    for i, x in enumerate(old):
        for t in range(start[i]):
            K[table[i][t // page], t % page] = x[t, :Hkv]
            V[table[i][t // page], t % page] = x[t, Hkv:]
    K, V, lens, count = K.cuda(), V.cuda(), i32(start), i32([len(free)])
    tab, fr, q = i32(table), i32(free), i32([1] * n)
    cu, slots, pos = i32([0] * (n + 1)), i32([0] * n), i32([0] * n)
    x, O = new[0].cuda(), torch.zeros(n, Hq, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(n, Hq, device="cuda")
    p = api.make_paged_params(n, width, n_pages, page, n_tokens=n, Hq=Hq, Hkv=Hkv, window=window,
                              n_sink=n_sink)
    ws = api.alloc_paged_workspace(p)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            api.paged_tables(p, lens, q, fr, count, tab, cu, lens, slots, pos, count)
            api.paged_append(p, slots, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], K, V)
            api.paged_attn(p, x[:, :Hq], K, V, tab, cu, lens, O, lse, ws)
    got = []
    for step in range(steps):
        x.copy_(new[step])
        graph.replay()
        got.append((f64(O), f64(lse)))
    torch.cuda.synchronize()
    assert api.get_status() == 0 and count.item() == 0 and lens.tolist() == [s + steps for s in start]
    a = f64(new)
    for i in range(n):
        kv = np.concatenate([f64(old[i]), a[:, i, Hq:]])
        ref = wo.attention(a[:, i, :Hq], kv[:, :Hkv], kv[:, Hkv:], start[i] + np.arange(steps), window,
                           n_sink)
        check(np.stack([o[i] for o, _ in got]), np.stack([ls[i] for _, ls in got]), ref, start[i] + steps)


# ---------------------------------------------------------------------------
# refusals (no GPU needed)
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kw,code", [
    (dict(page_size=48), host_api.ERR_UNSUPPORTED), (dict(page_size=256), host_api.ERR_UNSUPPORTED),
    (dict(page_size=0), host_api.ERR_UNSUPPORTED), (dict(head_dim=64), host_api.ERR_UNSUPPORTED),
    (dict(Hq=6, Hkv=2), host_api.ERR_UNSUPPORTED), (dict(Hq=5, Hkv=2), host_api.ERR_INVALID_ARG),
    (dict(n_seqs=-1), host_api.ERR_INVALID_ARG), (dict(n_seqs=8193), host_api.ERR_UNSUPPORTED),
    (dict(n_tokens=-1), host_api.ERR_INVALID_ARG), (dict(n_pages=0), host_api.ERR_INVALID_ARG),
    (dict(max_pages=0), host_api.ERR_INVALID_ARG), (dict(window=-1), host_api.ERR_INVALID_ARG),
    (dict(n_sink=-1), host_api.ERR_INVALID_ARG), (dict(scale=-1.0), host_api.ERR_INVALID_ARG),
    (dict(scale=float("nan")), host_api.ERR_INVALID_ARG),
    (dict(n_pages=1 << 25), host_api.ERR_UNSUPPORTED),       # slots past 32 bits
    (dict(max_pages=1 << 23), host_api.ERR_UNSUPPORTED),
])
def test_paged_bad_params(kw, code):
    lib = host_api.load()
    base = dict(n_seqs=2, max_pages=4, n_pages=8, page_size=64, n_tokens=2, Hq=4, Hkv=2)
    base.update(kw)
    P = ctypes.byref(host_api.make_paged_params(**base))
    assert lib.infllmv2_paged_tables(P, *[FAKE] * 10, None) == code
    assert lib.infllmv2_paged_append(P, FAKE, FAKE, 4096, FAKE, 4096, FAKE, FAKE, None) == code
    assert lib.infllmv2_paged_attn(P, FAKE, 4096, *[FAKE] * 8, 1 << 40, None) == code
    with pytest.raises(host_api.InfLLMV2Error):
        host_api.paged_workspace_bytes(host_api.make_paged_params(**base))


def test_paged_bad_pointers_strides_and_workspace():
    lib = host_api.load()
    p = host_api.make_paged_params(2, 4, 8, 64, n_tokens=2, Hq=4, Hkv=2)
    P = ctypes.byref(p)
    attn = lambda q=FAKE, qs=512, o=FAKE, t=FAKE, w=FAKE, nb=1 << 40: lib.infllmv2_paged_attn(  # noqa: E731
        P, q, qs, FAKE, FAKE, t, FAKE, FAKE, o, FAKE, w, nb, None)
    assert attn(q=None) == host_api.ERR_INVALID_ARG
    assert attn(q=FAKE + 8) == host_api.ERR_UNSUPPORTED
    assert attn(qs=504) == host_api.ERR_INVALID_ARG       # rows would overlap
    assert attn(qs=516) == host_api.ERR_UNSUPPORTED       # not whole 16-byte pieces
    assert attn(o=FAKE + 16) == host_api.ERR_UNSUPPORTED
    assert attn(t=None) == host_api.ERR_INVALID_ARG
    assert attn(t=FAKE + 2) == host_api.ERR_UNSUPPORTED
    assert attn(w=None) == host_api.ERR_INVALID_ARG
    assert attn(nb=host_api.paged_workspace_bytes(p) - 1) == host_api.ERR_WORKSPACE
    app = lambda s=FAKE, k=FAKE, ks=256: lib.infllmv2_paged_append(  # noqa: E731
        P, s, k, ks, FAKE, 256, FAKE, FAKE, None)
    assert app(s=None) == host_api.ERR_INVALID_ARG
    assert app(s=FAKE + 1) == host_api.ERR_UNSUPPORTED
    assert app(k=FAKE + 4) == host_api.ERR_UNSUPPORTED
    assert app(ks=128) == host_api.ERR_INVALID_ARG
    tab = [FAKE] * 10
    for i in range(10):
        bad = list(tab)
        bad[i] = None
        assert lib.infllmv2_paged_tables(P, *bad, None) == host_api.ERR_INVALID_ARG
        bad[i] = FAKE + 2
        assert lib.infllmv2_paged_tables(P, *bad, None) == host_api.ERR_UNSUPPORTED
    # nothing to do
    none = ctypes.byref(host_api.make_paged_params(2, 4, 8, 64, n_tokens=0, Hq=4, Hkv=2))
    assert lib.infllmv2_paged_attn(none, None, 512, *[None] * 8, 0, None) == host_api.OK
    assert lib.infllmv2_paged_append(none, None, None, 256, None, 256, None, None, None) == host_api.OK


def test_paged_params_struct_layout_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("needs a C compiler")
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                          "infllmv2.h")
    names = [f[0] for f in host_api.PagedParams._fields_]
    src = tmp_path / "layout.c"
    body = "\n".join(f'printf("{n} %zu\\n", offsetof(infllmv2_paged_params, {n}));' for n in names)
    src.write_text(f'#include <stddef.h>\n#include <stdio.h>\n#include "{header}"\n'
                   f'int main(void) {{ printf("sizeof %zu\\n", sizeof(infllmv2_paged_params));\n'
                   f'{body} return 0; }}\n')
    subprocess.run(["gcc", "-std=c99", "-o", str(tmp_path / "x"), str(src)], check=True)
    out = dict(line.split() for line in subprocess.run([str(tmp_path / "x")], check=True, text=True,
                                                       capture_output=True).stdout.splitlines())
    assert int(out["sizeof"]) == ctypes.sizeof(host_api.PagedParams)
    for n in names:
        assert int(out[n]) == getattr(host_api.PagedParams, n).offset, n


@pytest.mark.parametrize("bad", ["cpu", "table", "pool", "rows"])
def test_paged_binding_refuses_wrong_tensors(bad):
    import torch
    bf = torch.bfloat16
    p = host_api.make_paged_params(2, 4, 8, 16, n_tokens=3, Hq=4, Hkv=2)
    K = torch.zeros(8, 16, 2, 128, dtype=bf)
    Q = torch.zeros(3, 4, 128, dtype=bf)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    table = z(2, 5) if bad == "table" else z(2, 4)
    if bad == "pool":
        K = K[:7]
    if bad == "rows":
        Q = torch.zeros(3, 128, 4, dtype=bf).transpose(1, 2)
    with pytest.raises(host_api.InfLLMV2Error):
        host_api.paged_attn(p, Q, K, K, table, z(3), z(2), torch.zeros(3, 4, 128, dtype=bf),
                            torch.zeros(3, 4), torch.zeros(16, dtype=torch.uint8))
