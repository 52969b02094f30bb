"""GPU tests of the page operators (accepted drafts, forks, resizes) against
their definitions entry by entry; whole numbers and bytes are equal."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_04_gb300 as pkv
from paged_kv_gqa_04_gb300 import _abi
from tests._spec import accept_reference, fork_reference, make_tree, resize_reference, run_tree, check_tree

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _table(r, counts, width, pool):
    perm, bt, at = r.permutation(pool), np.full((len(counts), width), -1, np.int32), 0
    for b, n in enumerate(counts):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt


# ---- caches of every kind ---------------------------------------------------------------------------------------

def _cache(r, kind, pages, P):
    """A device cache of random bytes, its layout, and its bytes as [pages, P, n] (token rows) on the host."""
    dims = {"bf16_hnd": (2, "HND", torch.bfloat16, 64), "bf16_nhd": (3, "NHD", torch.bfloat16, 128),
            "fp8_hnd": (1, "HND", torch.uint8, 128), "scales_hnd": (3, "HND", torch.uint8, 4),
            "scales_odd": (3, "HND", torch.uint8, 5), "ckv": (0, "HND", torch.uint8, 512),
            "kpe": (0, "HND", torch.bfloat16, 64), "view": (2, "HND", torch.bfloat16, 64),
            "view_nhd": (2, "NHD", torch.bfloat16, 64), "wide": (2, "HND", torch.uint8, 128)}[kind]
    H, layout, dt, W = dims
    shape = (pages, P, W) if H == 0 else (pages, H, P, W) if layout == "HND" else (pages, P, H, W)
    if kind.startswith("view"):   # one of two in a joined tensor
        base = torch.zeros((pages, 2) + shape[1:], dtype=dt, device="cuda")
        t = base[:, 1]
    elif kind == "wide":          # rows with a gap behind them
        base = torch.zeros(shape[:-1] + (W + 16,), dtype=dt, device="cuda")
        t = base[..., :W]
    else:
        t = base = torch.zeros(shape, dtype=dt, device="cuda")
    raw = torch.from_numpy(r.randint(0, 256, shape[:-1] + (W * t.element_size(),)).astype(np.uint8)).cuda()
    t.copy_(raw.view(dt))
    return t, base, layout


def _bytes(t, layout):
    x = t.contiguous().view(torch.uint8).cpu().numpy()
    if x.ndim == 4:
        if layout == "HND":
            x = x.transpose(0, 2, 1, 3)
        x = x.reshape(x.shape[0], x.shape[1], -1)
    return x.copy()


SETS = [("bf16_hnd",), ("bf16_nhd",), ("fp8_hnd", "scales_hnd"), ("scales_odd",), ("ckv", "kpe"), ("view",),
        ("view_nhd",), ("wide",), ("bf16_hnd",) * 70]


@pytest.mark.parametrize("kinds", SETS, ids=lambda k: f"{k[0]}x{len(k)}")
@pytest.mark.parametrize("P", [16, 64, 5])
def test_accept_moves_rows(kinds, P):
    r = np.random.RandomState(P + len(kinds))
    drafts = [0, 1, 7, 16, 31, 40, 5, 3]
    lens = np.array([9, 1, 7, 100, 63, 170, 64, 80], np.int32)
    counts = [-(-int(x) // P) for x in lens]
    pages = sum(counts) + 2
    bt = _table(r, counts, max(counts) + 1, pages)
    start = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32) + 3
    A = 12
    acc, n_acc = np.full((len(lens), A), -9, np.int32), np.zeros(len(lens), np.int32)
    for b, n in enumerate(drafts):
        k = min(n, A, r.randint(0, n + 1) if b else 0)
        acc[b, :k] = np.sort(r.permutation(n)[:k])
        n_acc[b] = k
    acc[3, :A] = np.arange(16 - A, 16)   # every row moves onto one that moves too
    n_acc[3] = A
    caches = [_cache(r, k, pages, P) for k in kinds]
    lay = caches[0][2]
    before = [_bytes(t, lay) for t, _, _ in caches]
    outside = [b.clone() for _, b, _ in caches]
    want, want_lens, flags = accept_reference(before, bt, lens, start, acc, n_acc, P)
    assert flags == 0
    err, out = _i32([0]), _i32(np.full(len(lens), -77))
    pkv.accept_drafts([t for t, _, _ in caches], _i32(bt), _i32(lens), _i32(start), _i32(acc), _i32(n_acc), out,
                      layout=lay, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert np.array_equal(out.cpu().numpy(), want_lens)
    for (t, base, _), w, old in zip(caches, want, outside):
        assert np.array_equal(_bytes(t, lay), w)
        if base.data_ptr() != t.data_ptr() or base.shape != t.shape:   # the bytes between the rows
            keep, now = old.clone(), base.clone()
            for x in (keep, now):
                (x[:, 1] if kinds[0].startswith("view") else x[..., :t.shape[-1]]).zero_()
            assert torch.equal(keep, now)


def test_accept_refuses_bad_lists_on_the_device():
    r = np.random.RandomState(2)
    lens = np.array([50, 50, 50, 50, 50, 3, 500, -1, 50, 50], np.int32)
    drafts = [8, 8, 8, 8, 8, 8, 8, 0, 8, 8]
    bt = _table(r, [4] * 10, 4, 50)
    start = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
    acc = np.tile(np.array([1, 3, 5, 7], np.int32), (10, 1))
    n_acc = np.array([4, 4, 4, 9, -1, 2, 2, 0, 5, 2], np.int32)
    acc[0] = [1, 1, 2, 3]      # not ascending
    acc[1] = [1, 3, 5, 8]      # past the drafts
    acc[2] = [-1, 3, 5, 7]
    bt[9, 2] = 50              # tokens 32..47 on a page outside the pool
    t, _, lay = _cache(r, "bf16_hnd", 50, 16)
    for b in range(10):
        one = slice(b, b + 1)
        before = _bytes(t, lay)
        want, want_lens, flags = accept_reference([before], bt[one], lens[one], start[b:b + 2], acc[one], n_acc[one], 16)
        err, out = _i32([0]), _i32([-77])
        pkv.accept_drafts([t], _i32(bt[one]), _i32(lens[one]), _i32(start[b:b + 2]), _i32(acc[one]), _i32(n_acc[one]),
                          out, layout=lay, err_flag=err)
        torch.cuda.synchronize()
        assert int(err.item()) == flags and flags, b
        assert np.array_equal(out.cpu().numpy(), want_lens) and np.array_equal(_bytes(t, lay), want[0])


def test_accept_without_caches_gives_lengths():
    err, out = _i32([0]), _i32([0, 0])
    pkv.accept_drafts([], _i32([[0, 1], [2, 3]]), _i32([20, 30]), _i32([0, 4, 9]), _i32([[1, 3], [0, 0]]), _i32([2, 0]),
                      out, err_flag=err)
    torch.cuda.synchronize()
    assert out.tolist() == [18, 25] and int(err.item()) == 0


def test_accept_without_caches_takes_any_page_size():
    """No cache says how long pages are: a length that 16-token pages would not hold is no error."""
    err, out = _i32([0]), _i32([0])
    pkv.accept_drafts([], _i32([[0, 1]]), _i32([100]), _i32([0, 4]), _i32([[1]]), _i32([1]), out, err_flag=err)
    torch.cuda.synchronize()
    assert out.tolist() == [97] and int(err.item()) == 0


# ---- resize --------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("B,pages,P,width", [(1, 1, 16, 1), (3, 40, 16, 12), (200, 3000, 16, 40), (7, 16385, 64, 2000),
                                             (1500, 60001, 16, 64), (64, 200003, 1, 5000), (16384, 40000, 16, 3)])
def test_resize_sequence_of_calls(B, pages, P, width):
    r = np.random.RandomState(B + pages)
    err = _i32([0])
    counts, refs = np.zeros(B, np.int32), np.zeros(pages, np.int32)
    refs[r.permutation(pages)[:pages // 7]] = 1       # pages that others hold
    bt = np.full((B, width), -1, np.int32)
    d = [_i32(x) for x in (bt, counts, refs)]
    offset = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")[1:] if B == 7 else None  # counts off 16 bytes
    if offset is not None:
        offset.copy_(d[2])
        d[2] = offset
    for step in range(6):
        share = (pages * P) // max(B, 1) if step < 3 else 3 * pages * P // (2 * max(B, 1))  # the last ones run out
        lens = r.randint(-1, max(2, min(share * 2, width * P) + 2), B).astype(np.int32)
        if step == 2:
            lens[:] = 0
        bt, counts, refs, flags = resize_reference(bt, counts, lens, refs, P)
        err.zero_()
        pkv.resize_sequences(d[0], d[1], _i32(lens), d[2], P, err_flag=err)
        torch.cuda.synchronize()
        assert int(err.item()) == flags, step
        for x, y in zip(d, (bt, counts, refs)):
            assert np.array_equal(x.cpu().numpy(), y), step


def test_resize_flags_contradictions():
    bt = np.array([[0, 1, 2], [3, 9, -1], [4, 5, 6], [7, 7, -1], [-1, -1, -1]], np.int32)
    counts = np.array([3, 2, 4, 2, 0], np.int32)                    # row 2 has more than its width
    refs = np.array([1, 1, 0, 1, 1, 1, 1, 1, 0], np.int32)          # page 2 is counted nowhere, page 9 does not exist
    lens = np.array([0, 0, 0, 0, 64], np.int32)
    b2, c2, r2, flags = resize_reference(bt, counts, lens, refs, 16)
    d, err = [_i32(x) for x in (bt, counts, refs)], _i32([0])
    pkv.resize_sequences(d[0], d[1], _i32(lens), d[2], 16, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == flags == _abi.FLAG_PAGE_RANGE | _abi.FLAG_PAGE_STATE | _abi.FLAG_SEQ_LEN_RANGE
    for x, y in zip(d, (b2, c2, r2)):
        assert np.array_equal(x.cpu().numpy(), y)


def test_resize_of_nothing_and_of_an_empty_pool():
    err = _i32([0])
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    pkv.resize_sequences(torch.empty((0, 4), dtype=torch.int32, device="cuda"), e, e, _i32([0, 0]), err_flag=err)
    bt, c = _i32([[-1, -1]]), _i32([0])
    pkv.resize_sequences(bt, c, _i32([5]), e, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == _abi.FLAG_POOL_EMPTY and c.tolist() == [0] and bt.tolist() == [[-1, -1]]


def test_resize_of_the_widest_tables():
    """Rows of 2^26 entries (as many as there may be); one gives pages back, one cannot have that many."""
    width, err = 1 << 26, _i32([0])
    bt = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    bt[0, :20] = torch.arange(20, dtype=torch.int32)
    bt[2, 0] = 30
    counts, refs = _i32([20, 0, 1]), _i32([1] * 20 + [0] * 10 + [1])
    pkv.resize_sequences(bt, counts, _i32([3, width, -1]), refs, 1, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == _abi.FLAG_POOL_EMPTY and counts.tolist() == [3, 0, 1]
    assert refs.tolist() == [1] * 3 + [0] * 27 + [1]
    assert bt[0, :5].tolist() == [0, 1, 2, -1, -1] and int((bt >= 0).sum()) == 4


@pytest.mark.parametrize("every", [1, 3, 40])
def test_resize_where_few_rows_grow(every):
    """Ranks whose owners lie far apart: only every so-many-th row takes pages."""
    B, pages, P, width = 3000, 20000, 16, 8
    r = np.random.RandomState(every)
    refs = (r.rand(pages) < 0.3).astype(np.int32)
    bt, counts = np.full((B, width), -1, np.int32), np.zeros(B, np.int32)
    lens = np.where(np.arange(B) % every == every - 1, r.randint(1, width * P + 1, B), -1).astype(np.int32)
    d, err = [_i32(x) for x in (bt, counts, refs)], _i32([0])
    bt, counts, refs, flags = resize_reference(bt, counts, lens, refs, P)
    pkv.resize_sequences(d[0], d[1], _i32(lens), d[2], P, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == flags
    for x, y in zip(d, (bt, counts, refs)):
        assert np.array_equal(x.cpu().numpy(), y)


# ---- fork ----------------------------------------------------------------------------------------------------------

def _fork(kinds, P, pages, bt, counts, lens, forks, refs, r):
    caches = [_cache(r, k, pages, P) for k in kinds]
    lay = caches[0][2]
    before = [_bytes(t, lay) for t, _, _ in caches]
    want = fork_reference(before, bt, counts, lens, forks, refs, P)
    d, err = [_i32(x) for x in (bt, counts, lens, refs)], _i32([0])
    copies = _i32(np.full((len(forks), 2), 55))
    pkv.fork_sequences([t for t, _, _ in caches], d[0], d[1], d[2], _i32(forks), d[3], copies, layout=lay, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == want[6]
    for x, y, name in zip(d + [copies], want[1:6], ("tables", "counts", "lens", "refs", "copies")):
        assert np.array_equal(x.cpu().numpy(), y), name
    for (t, _, _), y in zip(caches, want[0]):
        assert np.array_equal(_bytes(t, lay), y)
    return want[6]


@pytest.mark.parametrize("kinds", SETS, ids=lambda k: f"{k[0]}x{len(k)}")
def test_fork_shares_and_copies(kinds):
    r = np.random.RandomState(len(kinds))
    lens = np.array([33, 16, 0, 5, 100] + [0] * 6, np.int32)
    counts = np.array([3, 1, 0, 1, 8] + [0] * 6, np.int32)   # the last one holds a page more than its tokens need
    pages = 40
    bt = _table(r, counts, 9, pages)
    refs = np.zeros(pages, np.int32)
    refs[bt[bt >= 0]] = 1
    forks = np.array([[0, 5], [1, 6], [-1, 7], [4, 8], [0, 9], [2, 10]], np.int32)
    assert _fork(kinds, 16, pages, bt, counts, lens, forks, refs, r) == 0


@pytest.mark.parametrize("n,pages,P", [(1, 30000, 16), (1000, 20001, 16), (16384, 17000, 4)])
def test_fork_in_bulk(n, pages, P):
    r = np.random.RandomState(n)
    parents = 20
    lens = np.concatenate([r.randint(0, 5000 if n == 1 else 60, parents), np.zeros(n)]).astype(np.int32)
    counts = -(-lens // P)
    bt = _table(r, counts, int(counts.max()) + 1, pages)
    refs = np.zeros(pages, np.int32)
    refs[bt[bt >= 0]] = 1
    refs[r.permutation(pages)[:pages // 3]] += 1
    forks = np.stack([r.randint(0, parents, n), parents + r.permutation(n)], 1).astype(np.int32)
    flags = _fork(("scales_hnd",), P, pages, bt, counts, lens, forks, refs, r)
    assert flags == (_abi.FLAG_POOL_EMPTY if n == 16384 else 0)


def test_fork_refuses_contradictions():
    r = np.random.RandomState(1)
    lens = np.array([33, 16, 40, -2, 20, 0, 0, 0, 0, 0, 0, 0], np.int32)
    counts = np.array([3, 1, 2, 1, 2, 0, 0, 0, 0, 0, 0, 0], np.int32)   # row 2 holds too few pages
    bt = _table(r, counts, 3, 20)
    refs = np.zeros(20, np.int32)
    refs[bt[bt >= 0]] = 1
    bt[4, 1] = 20                                                         # a last page outside the pool
    forks = np.array([[0, 5], [1, 5], [2, 6], [3, 7], [0, 1], [12, 8], [0, 12], [0, -1], [4, 9], [5, 10], [0, 10],
                      [0, 11]], np.int32)
    flags = _fork(("bf16_hnd",), 16, 20, bt, counts, lens, forks, refs, r)
    assert flags == _abi.FLAG_PAGE_STATE | _abi.FLAG_SEQ_LEN_RANGE | _abi.FLAG_PAGE_RANGE


def test_fork_carries_a_bad_shared_entry_over():
    r = np.random.RandomState(3)
    bt = np.array([[2, 99, 1], [-1, -1, -1]], np.int32)
    refs = np.array([0, 1, 1, 0], np.int32)
    flags = _fork(("fp8_hnd",), 16, 4, bt, np.array([3, 0], np.int32), np.array([48, 0], np.int32),
                  np.array([[0, 1]], np.int32), refs, r)
    assert flags == _abi.FLAG_PAGE_RANGE


# ---- the step as it is used -----------------------------------------------------------------------------------------

@pytest.mark.parametrize("captured", [False, True])
def test_speculative_steps_end_to_end(captured):
    """Two layers, four sequences, several steps: pages taken, drafted tokens
    written and attended to, some accepted, pages returned; after every step
    the cache holds the accepted tokens' rows and the attention agrees with
    float64. Then the sequences are forked and the children go on alone."""
    r = np.random.RandomState(4)
    Hq, Hkv, D, N, A, rows, width, pages, layers = 8, 2, 128, 7, 7, 6, 24, 120, 2
    lens = np.array([5, 40, 16, 90], np.int32)
    B, dev = 4, "cuda"
    caches = [torch.zeros((pages, Hkv, 16, D), dtype=torch.bfloat16, device=dev) for _ in range(2 * layers)]
    bt, counts = torch.full((rows, width), -1, dtype=torch.int32, device=dev), torch.zeros(rows, dtype=torch.int32, device=dev)
    refs, err = torch.zeros(pages, dtype=torch.int32, device=dev), _i32([0])
    cos_sin = torch.randn((400, D), device=dev)
    keys = [[] for _ in range(B)]                       # the tokens each sequence is to hold, layer by layer
    lens_a, lens_b = _i32(np.concatenate([lens, [0, 0]])), _i32([0] * rows)
    pkv.resize_sequences(bt, counts, lens_a, refs, 16, err_flag=err)

    def tokens(n):
        return [torch.randn((n, Hkv, D), device=dev).to(torch.bfloat16) for _ in range(2 * layers)]

    def write(x, pos, rows_of):
        page = bt[rows_of.long(), (pos // 16).long()]
        slots = (page * 16 + pos % 16).to(torch.int32)
        for i in range(layers):
            pkv.rope_kv_write(None, x[2 * i], x[2 * i + 1], pos, cos_sin, caches[2 * i], caches[2 * i + 1], slots,
                              err_flag=err)
    for b in range(B):
        x = tokens(int(lens[b]))
        write(x, torch.arange(int(lens[b]), dtype=torch.int32, device=dev),
              torch.full((int(lens[b]),), b, device=dev))
        keys[b] = [_held(caches, bt, b, range(int(lens[b])))]
    q_start = _i32(np.arange(B + 1) * N)
    grown, accepted, n_acc = _i32([0] * rows), _i32(np.zeros((B, A))), _i32([0] * B)
    s = make_tree([16] * B, [N] * B, Hq, Hkv, D, seed=20)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = torch.empty(pkv.tree_decode_workspace(B * N, Hq, D, sms), dtype=torch.uint8, device=dev)
    x = tokens(B * N)
    pos, row_of = _i32(np.zeros(B * N)), torch.arange(B, device=dev).repeat_interleave(N)

    def part_one():
        grown.copy_(lens_a + N)
        grown[B:] = -1
        pkv.resize_sequences(bt, counts, grown, refs, 16, err_flag=err)
        pos.copy_((lens_a[:B, None] + torch.arange(N, device=dev)).reshape(-1))
        write(x, pos, row_of)
        for i in range(layers):
            run_tree(dict(s, k=caches[2 * i], v=caches[2 * i + 1], bt=bt[:B], seq_lens=grown[:B], q_start=q_start,
                          ws=ws, err=err, out=outs[i], lse=lses[i]))
        pkv.accept_drafts(caches, bt[:B], grown[:B], q_start, accepted, n_acc, lens_b[:B], err_flag=err)
        lens_b[B:] = -1
        pkv.resize_sequences(bt, counts, lens_b, refs, 16, err_flag=err)
        lens_a[:B] = lens_b[:B]
    outs, lses = [torch.empty_like(s["out"]) for _ in range(layers)], [torch.empty_like(s["lse"]) for _ in range(layers)]
    graph = None
    for step in range(5):
        old = lens_a.tolist()
        acc = np.zeros((B, A), np.int32)
        k = r.randint(0, A + 1, B).astype(np.int32)
        for b in range(B):
            acc[b, :k[b]] = np.sort(r.permutation(N)[:k[b]])
        accepted.copy_(_i32(acc))
        n_acc.copy_(_i32(k))
        for t in x:
            t.copy_(torch.randn(t.shape, device=dev))
        if captured and graph is None:
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                part_one()
        graph.replay() if captured else part_one()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert lens_a.tolist()[:B] == [o + int(n) for o, n in zip(old, k)]
        want = [-(-n // 16) for n in lens_a.tolist()[:B]]
        assert counts.tolist()[:B] == want and int(refs.sum()) == sum(want) and int(refs.max()) == 1
        # the accepted rows, as single writes of these tokens at their drafted positions give them
        ref = [torch.zeros_like(c) for c in caches]
        flat = (torch.arange(B * N, device=dev) // 16 * 16 + torch.arange(B * N, device=dev) % 16).to(torch.int32)
        for i in range(layers):
            pkv.rope_kv_write(None, x[2 * i], x[2 * i + 1], pos, cos_sin, ref[2 * i], ref[2 * i + 1], flat)
        for b in range(B):
            at = [b * N + int(j) for j in acc[b, :k[b]]]
            keys[b].append([c.permute(0, 2, 1, 3).reshape(-1, Hkv, D)[at] for c in ref])
            now = _held(caches, bt, b, range(lens_a.tolist()[b]))
            for c in range(2 * layers):
                assert torch.equal(now[c], torch.cat([part[c] for part in keys[b]]))
    # fork rows 1 and 3, then a chain of tokens on the children alone
    copies = _i32(np.zeros((2, 2)))
    counts[B:] = 0
    pkv.fork_sequences(caches, bt, counts, lens_a, _i32([[1, 4], [3, 5]]), refs, copies, err_flag=err)
    lens = lens_a.tolist()
    assert lens[4] == lens[1] and lens[5] == lens[3]
    parents = [_held(caches, bt, b, range(lens[b])) for b in (1, 3)]
    up = _i32([-1] * B + [lens[4] + 3, lens[5] + 20])
    pkv.resize_sequences(bt, counts, up, refs, 16, err_flag=err)
    pos2 = _i32(list(range(lens[4], lens[4] + 3)) + list(range(lens[5], lens[5] + 20)))
    write(tokens(23), pos2, torch.tensor([4] * 3 + [5] * 20, device=dev))
    torch.cuda.synchronize()
    for b, p in zip((1, 3), parents):
        for c, y in zip(_held(caches, bt, b, range(lens[b])), p):
            assert torch.equal(c, y)                 # the parents are as they were
    for b, p in zip((4, 5), parents):
        for c, y in zip(_held(caches, bt, b, range(lens[b])), p):
            assert torch.equal(c, y)
    t = make_tree([3, 20], [3, 20], Hq, Hkv, D, seed=21, mask="chain")
    t.update(k=caches[2], v=caches[3], bt=bt[B:].contiguous(), seq_lens=up[B:].contiguous(), err=err)
    run_tree(t)
    check_tree(t)
    pkv.resize_sequences(bt, counts, _i32([0] * rows), refs, 16, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and int(refs.abs().sum()) == 0 and bool((bt == -1).all())


def _held(caches, bt, b, positions):
    """The rows of the given positions of row b, per cache, [n, Hkv, D]."""
    p = torch.tensor(list(positions), dtype=torch.long, device="cuda")
    return [c[bt[b][p // 16].long(), :, p % 16].clone() for c in caches]
