"""stem_cache_extend on the GPU: page tables, slot maps, positions and tree masks
equal to the oracle's, word for word."""

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C

pytestmark = pytest.mark.gpu

b = pytest.importorskip("block_sparse_attention_stem_b200.binding")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def tree_parents(rng, new):
    out = []
    for n in new:
        out += [-1 if i == 0 or rng.random() < 0.1 else int(rng.integers(max(0, i - 6), i)) for i in range(max(n, 0))]
    return np.array(out, dtype=np.int32)


def run(table, ps, pages, cache, new, held, free, cursor, T, parents=None, words=0, out=None):
    t = dev(table)
    r = b.stem_cache_extend(t, ps, pages, dev(cache), dev(new), dev(held), dev(free), dev([cursor]), T,
                            parents=None if parents is None else dev(parents), mask_words=words, out=out)
    return t, r, b.stem_read_device_status(r.ws)


def check(table, ps, pages, cache, new, held, free, cursor, T, parents=None, words=0):
    ref = C.extend(table, ps, pages, cache, new, held, free, cursor, T, parents, words)
    t, r, status = run(table, ps, pages, cache, new, held, free, cursor, T, parents, words)
    for name, got in (("table", t), ("held", r.held), ("cu", r.cu_seqlens), ("kv", r.kv_lens), ("slots", r.slots),
                      ("positions", r.positions)):
        assert np.array_equal(got.cpu().numpy(), ref[name]), name
    assert int(r.cursor) == ref["cursor"]
    if parents is not None:
        assert np.array_equal(r.mask.cpu().numpy().view(np.uint32), ref["mask"])
    assert (status == 0) == (not ref["status"])
    assert status in ({0} if not ref["status"] else {dict(bad=8, pages=9)[x] for x in ref["status"]})


def setup(rng, S, ps, cache_hi, new_lo, new_hi, spare=True):
    cache, new = rng.integers(0, cache_hi + 1, S), rng.integers(new_lo, new_hi + 1, S)
    held = -(-cache // ps) + (rng.integers(0, 2, S) if spare else 0)
    width = int(max(held.max(), (-(-(cache + new) // ps)).max(), 1)) + 1
    pages = int(held.sum() + (-(-(cache + new) // ps)).sum()) + 8
    order = rng.permutation(pages)
    table = np.full((S, width), -7)  # what is not extended stays as it was
    o = 0
    for s in range(S):
        table[s, :held[s]] = order[o:o + held[s]]
        o += held[s]
    return cache, new, held, table, pages, order[o:]


@pytest.mark.parametrize("S,ps,cache_hi,new_lo,new_hi", [
    (1, 64, 0, 1, 1), (1, 64, 200, 0, 0), (3, 64, 64, 0, 1), (7, 128, 1000, 1, 1), (33, 192, 500, 0, 70),
    (255, 64, 3000, 1, 9), (1024, 64, 300, 0, 3), (1025, 64, 300, 0, 3), (2500, 256, 2000, 1, 4), (8192, 64, 100, 0, 2),
    (2, 64, 0, 20000, 30000), (4, 128, 777, 1, 9000)])
def test_equals_the_oracle(S, ps, cache_hi, new_lo, new_hi):
    rng = np.random.default_rng(S + ps)
    cache, new, held, table, pages, free = setup(rng, S, ps, cache_hi, new_lo, new_hi)
    T = int(new.sum()) + int(rng.integers(0, 40))  # a padded batch: entries behind the last token
    check(table, ps, pages, cache, new, held, free, 1 if len(free) > 1 else 0, T)


@pytest.mark.parametrize("S,new_lo,new_hi,words", [(1, 1, 1, 1), (1, 64, 64, 2), (5, 0, 33, 2), (64, 17, 63, 2),
                                                   (3, 200, 256, 8), (300, 1, 40, 3)])
def test_trees_equal_the_oracle(S, new_lo, new_hi, words):
    rng = np.random.default_rng(S + new_hi)
    cache, new, held, table, pages, free = setup(rng, S, 64, 900, new_lo, new_hi)
    T = int(new.sum()) + 3
    parents = np.concatenate([tree_parents(rng, new), np.full(3, 99)])  # what is behind the last token is not read
    check(table, 64, pages, cache, new, held, free, 0, T, parents, words)


def test_a_chain_of_parents_is_the_plain_step_with_a_causal_mask():
    n = 96
    t, r, status = run([[0, 1, 2, -1]], 64, 8, [100], [n], [2], [5, 6, 7], 0, n, np.arange(n) - 1, 3)
    assert status == 0
    assert r.positions.tolist() == list(range(100, 100 + n))
    bits = np.unpackbits(r.mask.cpu().numpy().view(np.uint8), axis=1, bitorder="little")
    assert np.array_equal(bits, np.tri(n, dtype=np.uint8))


def test_out_of_pages_and_rows_that_are_too_short():
    rng = np.random.default_rng(5)
    cache, new, held, table, pages, free = setup(rng, 40, 64, 500, 100, 400, spare=False)
    T = int(new.sum())
    check(table, 64, pages, cache, new, held, free[:17], 2, T)     # the list ends in the middle of a sequence
    check(table, 64, pages, cache, new, held, free[:0], 0, T)      # no list at all
    check(table[:, :5], 64, pages, cache, new, np.minimum(held, 5), free, 0, T)  # rows of five pages


@pytest.mark.parametrize("what", ["negative", "held", "cursor", "tokens", "free page", "held page", "parent", "words"])
def test_values_out_of_range_are_reported_and_stay_inside_the_arrays(what):
    rng = np.random.default_rng(6)
    cache, new, held, table, pages, free = setup(rng, 20, 64, 500, 3, 60, spare=False)
    T, cur, parents, words = int(new.sum()), 0, None, 0
    held, free = held.copy(), free.copy()
    if what == "negative":
        cache[3], new[5] = -4, -9
        held[3] = 0
    elif what == "held":
        held[4], held[7] = -2, 10 ** 6
    elif what == "cursor":
        cur = len(free) + 5
    elif what == "tokens":
        T -= 25
    elif what == "free page":
        free[2], free[4] = -3, pages + 9
    elif what == "held page":
        held[cache % 64 == 0] += 0
        s = int(np.argmax(cache % 64 > 0))
        table[s, cache[s] // 64] = pages  # the page that the next token would go to
    elif what == "parent":
        parents, words = tree_parents(rng, new), 2
        parents[1], parents[10] = 1, -2
    else:
        parents, words = tree_parents(rng, new), 1
        assert new.max() > 32
    check(table, 64, pages, cache, new, held, free, cur, T, parents, words)


def test_a_captured_step_advances_its_own_state():
    """held, cursor and the lengths written over the inputs, replayed: one token per step."""
    S, ps, steps = 5, 64, 150
    cache, new, held = dev([0, 63, 10, 64, 127]), dev([1] * S), dev([0, 1, 1, 1, 2])
    table = dev(np.full((S, 8), -1))
    table[1, 0], table[2, 0], table[3, 0], table[4, 0], table[4, 1] = 40, 41, 42, 43, 44
    ref_table, ref_held, ref_cache, cur = table.cpu().numpy(), held.cpu().numpy(), cache.cpu().numpy(), 0
    free, cursor = dev(np.arange(30)), dev([0])
    i32 = dict(dtype=torch.int32, device="cuda")
    out = b.CacheStep(held, cursor, torch.empty(S + 1, **i32), cache, torch.empty(S, **i32), torch.empty(S, **i32), None,
                      torch.empty(256, dtype=torch.uint8, device="cuda"))
    call = lambda: b.stem_cache_extend(table, ps, 64, cache, new, held, free, cursor, S, out=out)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(steps):
        graph.replay()
        r = C.extend(ref_table, ps, 64, ref_cache, [1] * S, ref_held, list(range(30)), cur, S)
        ref_table, ref_held, ref_cache, cur = r["table"], r["held"], r["kv"], r["cursor"]
        assert np.array_equal(out.slots.cpu().numpy(), r["slots"])
    assert np.array_equal(table.cpu().numpy(), ref_table) and np.array_equal(held.cpu().numpy(), ref_held)
    assert np.array_equal(cache.cpu().numpy(), ref_cache) and int(cursor) == cur
    assert b.stem_read_device_status(out.ws) == 0


def test_steps_of_many_sequences_from_two_threads():
    """Steps of different sizes enqueued at the same time, both past 48 KB of shared memory."""
    import ctypes
    import threading

    codes, keep = set(), []

    def work(S, stream):
        rng = np.random.default_rng(S)
        cache, new, held, table, pages, free = setup(rng, S, 64, 100, 1, 1, spare=False)
        ref = C.extend(table, 64, pages, cache, new, held, free, 0, S)
        with torch.cuda.stream(stream):
            t, ins = dev(table), [dev(x) for x in (cache, new, held, free, [0])]
            outs = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (S, 1, S + 1, S, S, S)]
            ws = torch.empty(256, dtype=torch.uint8, device="cuda")
        desc = b.StemCacheStep(S, S, 64, pages, t.shape[1], len(free), 0, *[x.data_ptr() for x in ins], None)
        args = [ctypes.byref(desc), t.data_ptr(), *[x.data_ptr() for x in outs], None, ws.data_ptr(), 256, stream.cuda_stream]
        keep.append((t, ins, outs, ws, desc, ref))
        return lambda: codes.update(b.LIB.stem_cache_extend(*args) for _ in range(4000))

    threads = [threading.Thread(target=work(S, torch.cuda.Stream())) for S in (8192, 3500)]
    torch.cuda.synchronize()
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert codes == {b.STEM_OK}
    for t, _, outs, _, _, ref in keep:
        assert np.array_equal(t.cpu().numpy(), ref["table"]) and np.array_equal(outs[4].cpu().numpy(), ref["slots"])


@pytest.mark.parametrize("cursor", [-1, 45])
def test_a_step_without_pages_says_so_whatever_else_is_wrong(cursor):
    """OUT_OF_PAGES is the status of a step that also has values out of range, every time."""
    rng = np.random.default_rng(8)
    cache, new, held, table, pages, free = setup(rng, 300, 64, 500, 50, 100, spare=False)
    T, cache = int(new.sum()), cache.copy()
    cache[[0, 150, 299]] = -5
    ref = C.extend(table, 64, pages, cache, new, held, free[:40], cursor, T)
    assert ref["status"] == {"bad", "pages"}
    for _ in range(20):
        _, r, status = run(table, 64, pages, cache, new, held, free[:40], cursor, T)
        assert status == 9
    assert np.array_equal(r.slots.cpu().numpy(), ref["slots"])
