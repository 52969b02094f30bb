"""GPU tests of the page operators as programs use them: from several host
threads, with pages that sequences share, and with the rotary positions of a
tree of drafted tokens."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import paged_kv_gqa_04_gb300 as pkv
from paged_kv_gqa_04_gb300 import _abi
from tests._spec import resize_reference

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def test_two_host_threads_resize_batches_of_different_sizes():
    """Two threads, a stream and a pool each: 16384 rows (the largest shared memory there is, returns by a kernel of
    their own) and 3 rows, at the same time. No call fails, and both pools end as the calls one by one give."""
    calls, failed = 2000, []

    def state(B, width, pages, seed):
        r = np.random.RandomState(seed)
        lens = [r.randint(0, 16 * width + 1, B).astype(np.int32) for _ in range(2)]
        bt, counts, refs = np.full((B, width), -1, np.int32), np.zeros(B, np.int32), np.zeros(pages, np.int32)
        want = (bt, counts, refs)
        d = [_i32(x) for x in want]
        for x in lens:                     # every later pair of calls starts from the same counts
            want = resize_reference(*want[:2], x, want[2], 16)[:3]
        return d, [_i32(x) for x in lens], want

    def work(d, lens, stream, err, gate):
        try:
            b = [pkv.bind(x) for x in d + lens + [err]]
            gate.wait()
            for i in range(calls):
                pkv.resize_sequences(b[0], b[1], b[3 + i % 2], b[2], 16, err_flag=b[5], stream=stream)
        except Exception as e:             # noqa: BLE001 (a failed call is what this looks for)
            failed.append(repr(e))
    sets = [state(16384, 4, 70000, 1), state(3, 4, 20000, 2)]
    errs = [_i32([0]), _i32([0])]
    torch.cuda.synchronize()
    gate = threading.Barrier(2)
    threads = [threading.Thread(target=work, args=(s[0], s[1], torch.cuda.Stream(), e, gate)) for s, e in zip(sets, errs)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not failed, failed[0]
    assert [int(e.item()) for e in errs] == [0, 0]
    for d, lens, want in sets:
        assert np.array_equal(d[1].cpu().numpy(), want[1])
        held, refs = d[0][d[0] >= 0].cpu().numpy(), d[2].cpu().numpy()
        assert np.array_equal(np.bincount(held, minlength=len(refs)), refs) and refs.max() == 1


@pytest.mark.parametrize("pages", [40, 9000, 40000])
@pytest.mark.parametrize("count", [-1, -2, -5, -16384, -16385, -2 ** 31 + 16384])
def test_children_with_negative_page_counts_are_refused(count, pages):
    """page_counts[child] has to be 0; others are a contradiction, alike for all numbers of forks and CTAs. A row
    that is refused stays as it is, and so does its parent."""
    bt, lens = _i32([[3, 4], [-1, -1], [-1, -1], [-1, -1]]), _i32([20, 0, 0, 0])
    counts, refs, err = _i32([2, count, 0, count]), torch.zeros(pages, dtype=torch.int32, device="cuda"), _i32([0])
    refs[3:5] = 1
    cache = torch.randn((pages, 1, 16, 8), device="cuda")
    before = cache.clone()
    forks, copies = _i32([[0, 1], [0, 2], [0, 3], [0, 3]]), _i32(np.zeros((4, 2)))
    pkv.fork_sequences([cache], bt, counts, lens, forks, refs, copies, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pkv.FLAG_PAGE_STATE
    assert counts.tolist() == [2, count, 2, count] and lens.tolist() == [20, 0, 20, 0]
    assert copies.tolist() == [[-2, -2], [4, 0], [-2, -2], [-2, -2]]
    assert bt.tolist() == [[3, 4], [-1, -1], [3, 0], [-1, -1]]
    before[0] = before[4]
    assert torch.equal(cache, before)
    assert refs[:5].tolist() == [1, 0, 0, 2, 1] and int(refs.sum()) == 4


@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_accepted_path_of_a_tree_is_what_one_token_at_a_time_leaves(layout):
    """Drafted token j of a tree is rotated at base + its depth (the position it has if its path is accepted) and
    stored at base + j. Every row's attention is then that of its path written token by token, and the cache
    behind an accepted path is byte for byte what those writes leave."""
    Hq, Hkv, D, base, pages = 8, 2, 128, 37, 6
    parent = [-1, -1, 0, 0, 2, 1, 2, 6, 3, 7]             # ten drafted tokens; -1 hangs below the context
    N = len(parent)
    depth = []
    for p in parent:
        depth.append(depth[p] + 1 if p >= 0 else 0)

    def path(j):
        return path(parent[j]) + [j] if j >= 0 else []
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def rnd(*s):
        return torch.randn(s, generator=g, device="cuda").bfloat16()
    q, k, v = rnd(N, Hq, D), rnd(base + N, Hkv, D), rnd(base + N, Hkv, D)   # the context's k and v, then the drafts'
    cs, err = torch.randn((64, D), generator=g, device="cuda"), _i32([0])
    shape = (pages, Hkv, 16, D) if layout == "HND" else (pages, 16, Hkv, D)
    table = np.array([4, 1, 5, 0], np.int32)

    def cache_of(rows, positions, stored, q=None):
        kc, vc = torch.zeros(shape, device="cuda").bfloat16(), torch.zeros(shape, device="cuda").bfloat16()
        slots = table[np.array(stored) // 16] * 16 + np.array(stored) % 16
        pkv.rope_kv_write(None, k[rows], v[rows], _i32(positions), cs, kc, vc, _i32(slots), layout=layout, err_flag=err)
        return kc, vc
    ctx = list(range(base))
    kc, vc = cache_of(ctx + [base + j for j in range(N)], ctx + [base + d for d in depth], ctx + [base + j for j in range(N)])
    qr = q.clone()
    scratch = [torch.zeros(shape, device="cuda").bfloat16() for _ in range(2)]
    pkv.rope_kv_write(qr, k[base:], v[base:], _i32([base + d for d in depth]), cs, *scratch,
                      _i32(np.arange(N)), layout=layout, err_flag=err)
    bits = [sum(1 << x for x in path(j)) for j in range(N)]
    out, lse = torch.zeros_like(q), torch.zeros((N, Hq), device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = torch.empty(pkv.tree_decode_workspace(N, Hq, D, sms), dtype=torch.uint8, device="cuda")
    bt = _i32(table[None])
    pkv.paged_tree_decode(qr, kc, vc, bt, _i32([base + N]), _i32([0, N]), _i32(np.array(bits)[:, None]), D ** -0.5, out, lse,
                          ws, layout=layout, err_flag=err)
    for j in range(N):
        p = path(j)
        L = base + len(p)
        ks, vs = cache_of(ctx + [base + x for x in p], list(range(L)), list(range(L)))
        op, lp = torch.empty((1, 2, Hq, D), device="cuda"), torch.empty((1, 2, Hq), device="cuda")
        o1, l1 = torch.empty((1, Hq, D), device="cuda").bfloat16(), torch.empty((1, Hq), device="cuda")
        pkv.paged_gqa_decode(qr[j:j + 1], ks, vs, bt, _i32([L]), D ** -0.5, 2, op, lp, layout=layout, err_flag=err)
        pkv.lse_merge(op, lp, o1, l1)
        # the same scores and weights but for the order of fp32 sums and 2^-16 of a weight (|v| < 5); then either
        # output is within half a step of bf16 of its value
        d = (out[j] - o1[0]).double().abs()
        assert bool((d <= 2 * 2.0 ** -8 * o1[0].double().abs() + 5 * 2.0 ** -13).all())
        assert bool(((lse[j] - l1[0]).abs() <= 2.0 ** -14).all())
        # the path accepted: in a copy of the cache, its rows moved together
        kj, vj, new = kc.clone(), vc.clone(), _i32([0])
        pkv.accept_drafts([kj, vj], bt, _i32([base + N]), _i32([0, N]), _i32([p]), _i32([len(p)]), new, layout=layout,
                          err_flag=err)
        assert new.tolist() == [L]
        for a, b in ((kj, ks), (vj, vs)):
            for t in range(L):
                page, off = int(table[t // 16]), t % 16
                x, y = (a[page, :, off], b[page, :, off]) if layout == "HND" else (a[page, off], b[page, off])
                assert torch.equal(x, y), (j, t)
    assert int(err.item()) == 0


def test_a_row_trimmed_into_a_shared_page_goes_on_as_a_fork():
    """A trim below the fork point leaves a row whose last page another one still reads. A fork of it gets a page of
    its own for the tokens to come, and the other sequence's tokens stay."""
    pages, err = 12, _i32([0])
    cache = torch.randn((pages, 1, 16, 8), device="cuda")
    bt, counts, lens = _i32(np.full((4, 4), -1)), _i32([0] * 4), _i32([40, 0, 0, 0])
    refs, copies = torch.zeros(pages, dtype=torch.int32, device="cuda"), _i32(np.zeros((1, 2)))
    pkv.resize_sequences(bt, counts, _i32([40, -1, -1, -1]), refs, 16, err_flag=err)
    pkv.fork_sequences([cache], bt, counts, lens, _i32([[0, 1]]), refs, copies, err_flag=err)
    assert bt[:2].tolist() == [[0, 1, 2, -1], [0, 1, 3, -1]] and refs[:4].tolist() == [2, 2, 1, 1]
    # row 0 back to 20 tokens, in the middle of page 1, which row 1 reads: it goes on as row 2
    pkv.resize_sequences(bt, counts, _i32([20, -1, -1, -1]), refs, 16, err_flag=err)
    lens[0] = 20
    assert bt[0].tolist() == [0, 1, -1, -1] and refs[:4].tolist() == [2, 2, 0, 1]
    pkv.fork_sequences([cache], bt, counts, lens, _i32([[0, 2]]), refs, copies, err_flag=err)
    pkv.resize_sequences(bt, counts, _i32([0, -1, 33, -1]), refs, 16, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and copies.tolist() == [[1, 2]]
    assert bt.tolist() == [[-1] * 4, [0, 1, 3, -1], [0, 2, 4, -1], [-1] * 4]
    assert refs[:5].tolist() == [2, 1, 1, 1, 1] and counts.tolist() == [0, 3, 3, 0] and lens.tolist() == [20, 40, 20, 0]
    assert torch.equal(cache[2], cache[1])                # tokens 16 .. 19 of row 2 (and what lies behind them)


@pytest.mark.parametrize("B,width", [(5000, 400), (1300, 1700)])
def test_rows_that_return_more_than_a_grid_takes_at_once(B, width):
    """More rows than SMs have warps for, and returns of several stretches of 256 entries each, bad ones among them."""
    r = np.random.RandomState(B)
    counts = r.randint(width // 2, width + 1, B).astype(np.int32)
    pages = int(counts.sum()) + 7
    bt = np.full((B, width), -1, np.int32)
    bt[np.arange(width) < counts[:, None]] = r.permutation(pages)[:counts.sum()]
    refs = np.zeros(pages, np.int32)
    refs[bt[bt >= 0]] = 1
    bt[3, 5], bt[7, 2] = pages, bt[7, 3]
    lens = (r.randint(0, width // 3, B) * 16).astype(np.int32)
    lens[[0, 3, 7]] = 0
    want = resize_reference(bt, counts, lens, refs, 16)
    d, err = [_i32(x) for x in (bt, counts, refs)], _i32([0])
    pkv.resize_sequences(d[0], d[1], _i32(lens), d[2], 16, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == want[3] == pkv.FLAG_PAGE_RANGE | pkv.FLAG_PAGE_STATE
    assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(d, want))


def test_an_empty_list_overlaps_nothing():
    """No accepted tokens at all (A = 0), wherever the list's pointer points: the new lengths' own memory here."""
    lens, start, none, err = _i32([20, 5, 3]), _i32([0, 4, 4, 7]), _i32([0, 0, 0]), _i32([0])
    bt, out = _i32(np.arange(6).reshape(3, 2)), _i32([7, 7, 7])
    empty = _abi.PkvTensor.from_buffer_copy(_abi._desc(bt).contents)
    empty.ptr, empty.shape[1] = out.data_ptr() + 4, 0
    d = [_abi._desc(x) for x in (bt, lens, start)]
    st = _abi.lib().pkv_accept_drafts(None, 0, 1, *d, ctypes.pointer(empty), _abi._desc(none), _abi._desc(out),
                                      err.data_ptr(), _abi._stream(None))
    torch.cuda.synchronize()
    assert st == _abi.PKV_OK and int(err.item()) == 0 and out.tolist() == [16, 5, 0]
