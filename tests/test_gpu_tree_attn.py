"""stem_tree_attn on the GPU against the fp64 oracle.

Bounds of one output element, with A = sum p |v| / sum p, L the number of keys and
e = (128 + 8) 2^-24 max sigma |q|.|k| the error of a logit (128 products summed in
fp32, and its scaling):
  * a weight is off by e (twice: its own logit and the normalisation), exp2 by
    2^-21, and P by 2^-15 (two bf16: the first cut off below p, the rest, at
    most 2^-7 p, rounded) or, e4m3 inputs, 2^-11 (f16; below its normal
    range 2^-25 absolute, against weights whose largest is at least 1/2);
  * the sums of L weights and products in fp32 by L 2^-24 each;
  * out rounds to bf16: 2^-8 |o|.
lse: e, L 2^-24, 2^-20 for exp2 and log2, and 2^-22 |lse| for its own arithmetic."""

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C
from oracle import stem_oracle as O

pytestmark = pytest.mark.gpu

b = pytest.importorskip("block_sparse_attention_stem_b200.binding")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


class Case:
    """Random queries, pages and masks of given lengths; unused pool rows are NaN."""

    def __init__(self, new, ctx, hq, hkv, fp8=False, ps=64, tree=False, words=None, seed=0, extra=0, scale=0.0, spread=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        self.new, self.kv, self.hq, self.hkv, self.fp8, self.ps, self.scale = new, [c + n for c, n in zip(ctx, new)], hq, hkv, fp8, ps, scale
        S, T = len(new), sum(new) + extra
        self.T, self.cu = T, [0] + list(np.cumsum(new))
        npg = [-(-k // ps) for k in self.kv]
        P = sum(npg) + 2
        order = rng.permutation(P)
        self.table = np.full((S, max(max(npg), 1) + 1), -1, dtype=np.int32)
        o = 0
        for s in range(S):
            self.table[s, :npg[s]] = order[o:o + npg[s]]
            o += npg[s]
        used = torch.zeros(P * ps, dtype=torch.bool, device="cuda")
        for s in range(S):
            used[self.rows(s)] = True
        self.qs = self.ks = self.vs = None
        if fp8:
            self.qs, self.ks, self.vs = (torch.rand(h, generator=g, device="cuda") * 0.01 + 0.005 for h in (hq, hkv, hkv))
        self.q = self._enc(torch.randn(T, hq, 128, generator=g, device="cuda") * spread, self.qs)
        self.k, self.v = (self._enc(torch.randn(P * ps, hkv, 128, generator=g, device="cuda"), sc).view(P, ps, hkv, 128)
                          for sc in (self.ks, self.vs))
        nan = 0x7F if fp8 else float("nan")
        for x in (self.k, self.v):
            x.view(P * ps, hkv, 128)[~used] = nan
        self.mask = None
        if tree:
            words = words or -(-max(new) // 32)
            m = np.zeros((T, words), dtype=np.uint32)
            for s in range(S):
                for i in range(new[s]):
                    row = m[self.cu[s] + i]
                    if i and i % 7:  # an ancestor's row and the token itself; every seventh starts afresh
                        row |= m[self.cu[s] + int(rng.integers(max(0, i - 4), i))]
                    if i // 32 < words:
                        row[i // 32] |= np.uint32(1 << (i % 32))
            self.mask = m

    def _enc(self, x, sc):
        if not self.fp8:
            return x.to(torch.bfloat16)
        return (x / sc[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def rows(self, s):
        u = np.arange(self.kv[s])
        return torch.from_numpy(self.table[s, u // self.ps].astype(np.int64) * self.ps + u % self.ps).cuda()

    def f64(self, x, sc):
        if not self.fp8:
            return x.double().cpu().numpy()
        return O.e4m3_bytes_to_f64(x.cpu().numpy()) * sc.double().cpu().numpy()[None, :, None]

    def oracle(self):
        kr, vr = ([self.f64(x.view(-1, self.hkv, 128)[self.rows(s)], sc) for s in range(len(self.new))]
                  for x, sc in ((self.k, self.ks), (self.v, self.vs)))
        return C.tree_attn(self.f64(self.q, self.qs), kr, vr, self.cu, self.kv, self.mask, self.scale)

    def gpu(self, max_seq_tokens=None, out=None, lse=None, ws=None, stream=None, tree=None):
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.cache = b.paged_kv(self.k, self.v, i32(self.table), self.ps)
        self.tree = b.make_tree(self.q, i32(self.cu), i32(self.kv), self.hkv,
                                mask=None if self.mask is None else i32(self.mask.view(np.int32)),
                                max_seq_tokens=max(self.new) if max_seq_tokens is None else max_seq_tokens,
                                q_scale=self.qs, k_scale=self.ks, v_scale=self.vs, softmax_scale=self.scale)
        out, lse, ws = b.stem_tree_attn(self.tree, self.cache, out=out, lse=lse, ws=ws, stream=stream)
        return out, lse, b.stem_read_device_status(ws, stream)

    def check(self, status=0, **kw):
        out, lse, st = self.gpu(**kw)
        assert st == status
        o, z, e = self.oracle()
        n = self.cu[-1]
        out, lse = out[:n].double().cpu().numpy(), lse[:, :n].double().cpu().numpy()
        assert np.array_equal(np.isneginf(lse), np.isneginf(z[:, :n]))
        L = max(self.kv)
        logit = 136 * 2.0 ** -24 * e["qk"][:n]
        w = 2 * logit + 2.0 ** -20 + (2.0 ** -10 if self.fp8 else 2.0 ** -15) + 2 * L * 2.0 ** -24
        tol = 2.0 ** -8 * np.abs(o[:n]) + w[..., None] * e["absav"][:n] + 1e-30
        if self.fp8:
            tol += (2 * L * 2.0 ** -25 * e["vmax"][:n])[..., None]
        assert np.all(np.abs(out - o[:n]) <= tol), float((np.abs(out - o[:n]) / tol).max())
        see = ~np.isneginf(lse)
        lz, zz = np.where(see, lse, 0), np.where(see, z[:, :n], 0)
        assert np.all(np.abs(lz - zz) <= logit.T + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * np.abs(zz))
        assert np.all(out[~see.T] == 0)
        return out, lse


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctx", [0, 1, 62, 63, 64, 127, 128, 300, 1000, 5001])
def test_single_tokens(ctx, fp8):
    Case([1], [ctx], 8, 2, fp8, seed=ctx).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (3, 1), (6, 2), (20, 4), (8, 1), (33, 1), (64, 1), (65, 1), (128, 1)])
def test_head_layouts(hq, hkv, fp8):
    Case([3, 1], [200, 77], hq, hkv, fp8, seed=hq).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,ctx", [(2, 0), (5, 60), (16, 48), (31, 33), (32, 1000), (33, 127), (63, 1), (64, 640),
                                   (65, 64), (100, 30), (256, 100)])
def test_trees(n, ctx, fp8):
    Case([n], [ctx], 4, 1, fp8, tree=True, seed=n).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,ctx", [(2, 0), (64, 0), (65, 3), (200, 500), (700, 129)])
def test_causal_chunks(n, ctx, fp8):
    Case([n], [ctx], 3, 1, fp8, seed=n).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ps", [64, 128, 192, 256])
def test_ragged_batches_and_page_sizes(ps, fp8):
    Case([1, 7, 0, 33, 2, 12, 1], [900, 0, 50, 63, 64, 1500, 191], 8, 2, fp8, ps=ps, tree=True, seed=ps).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_many_short_sequences(fp8):
    """Items of one unit, several per range, and more sequences than threads."""
    rng = np.random.default_rng(3)
    new = [int(x) for x in rng.integers(0, 3, 700)]
    new[17] = 40  # Q tiles of more than 64 rows have a single buffer
    Case(new, [int(x) for x in rng.integers(0, 70, 700)], 4, 2, fp8, seed=3).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_one_unit_items_with_full_tiles(fp8):
    """Many items of one unit whose Q tile fills the single buffer."""
    S = 400
    Case([32] * S, [0, 20, 32, 5] * (S // 4), 8, 2, fp8, tree=True, seed=4).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_large_logits(fp8):
    """The running reference moves often, and weights underflow."""
    Case([5, 1], [2000, 3000], 4, 2, fp8, seed=8, spread=12.0).check()
    Case([5, 1], [2000, 3000], 4, 2, fp8, seed=9, scale=1.5).check()


def test_more_tiles_than_ranges():
    c = Case([9700], [30], 4, 1, seed=10)
    out, lse, st = c.gpu()
    assert st == 0
    k = c.f64(c.k.view(-1, 1, 128)[c.rows(0)], None)
    v = c.f64(c.v.view(-1, 1, 128)[c.rows(0)], None)
    q = c.f64(c.q, None)
    for t in (0, 1, 31, 32, 5000, 9699):
        L = 30 + t + 1
        o, z, e = C.tree_attn(q[t:t + 1], [k[:L]], [v[:L]], [0, 1], [L])
        logit = 136 * 2.0 ** -24 * e["qk"]
        tol = 2.0 ** -8 * np.abs(o) + (2 * logit + 2.0 ** -14 + 2 * L * 2.0 ** -24)[..., None] * e["absav"]
        assert np.all(np.abs(out[t].double().cpu().numpy() - o[0]) <= tol[0])
        assert np.all(np.abs(lse[:, t].double().cpu().numpy() - z[:, 0]) <= logit[0] + L * 2.0 ** -24 + 2.0 ** -18)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_context_split_over_all_ranges(fp8):
    Case([4], [70000], 4, 1, fp8, tree=True, seed=11).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,hq", [(60, 5), (45, 3), (20, 7), (3, 5), (1, 13)])
def test_cut_items_of_odd_groups(n, hq, fp8):
    """Tiles of fewer than 128 rows, several of them, cut over many ranges."""
    Case([n, 1], [3000, 2000], hq, 1, fp8, tree=True, seed=n + hq).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_very_long_context(fp8):
    """700,000 keys: one sequence and KV head over every range; rows checked on the GPU in fp64."""
    L, hq = 700_001, 4
    g = torch.Generator("cuda").manual_seed(31)
    P = -(-L // 64)
    sc = [torch.full((h,), 0.01, device="cuda") for h in (hq, 1, 1)] if fp8 else [None] * 3
    x = [torch.randn(n, h, 128, generator=g, device="cuda") for n, h in ((1, hq), (P * 64, 1), (P * 64, 1))]
    enc = [(y / 0.01).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else y.to(torch.bfloat16) for y in x]
    dec = [y.view(torch.float8_e4m3fn).double() * float(s[0]) if fp8 else y.double() for y, s in zip(enc, sc)]
    perm = torch.randperm(P, generator=g, device="cuda")
    pools = [torch.empty_like(y).view(P, 64, 1, 128) for y in enc[1:]]
    for p, y in zip(pools, enc[1:]):
        p[perm] = y.view(P, 64, 1, 128)
    i32 = dict(dtype=torch.int32, device="cuda")
    tree = b.make_tree(enc[0], torch.tensor([0, 1], **i32), torch.tensor([L], **i32), 1, max_seq_tokens=1,
                       q_scale=sc[0], k_scale=sc[1], v_scale=sc[2])
    out, lse, ws = b.stem_tree_attn(tree, b.paged_kv(*pools, perm.to(torch.int32)[None].contiguous(), 64))
    assert b.stem_read_device_status(ws) == 0
    s = dec[0][0] @ dec[1][:L, 0].T / 128 ** 0.5
    z = torch.logsumexp(s, 1)
    p = torch.exp(s - z[:, None])
    o, av = p @ dec[2][:L, 0], p @ dec[2][:L, 0].abs()
    logit = 136 * 2.0 ** -24 * float((dec[0][0].abs() @ dec[1][:L, 0].abs().T).max()) / 128 ** 0.5
    # at most 296 pieces of 2400 keys, summed apart and then joined
    w = 2 * logit + 2.0 ** -20 + (2.0 ** -10 if fp8 else 2.0 ** -15) + 2 * (4800 + 296) * 2.0 ** -24
    assert torch.all((out[0].double() - o).abs() <= 2.0 ** -8 * o.abs() + w * av)
    assert torch.all((lse[:, 0].double() - z).abs() <= logit + 2.0 ** -18)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_whose_mask_leaves_nothing(fp8):
    c = Case([6, 40], [0, 0], 4, 2, fp8, tree=True, seed=12)
    c.mask[[1, 4, 9, 45]] = 0
    out, lse = c.check()
    assert np.all(np.isneginf(lse[:, [1, 4, 9, 45]])) and np.all(out[[1, 4, 9, 45]] == 0)


@pytest.mark.parametrize("fp8", [False, True])
def test_queries_without_any_key(fp8):
    c = Case([3, 2], [10, 5], 4, 2, fp8, seed=13)
    c.kv[1] = 0
    out, lse = c.check()
    assert np.all(np.isneginf(lse[:, 3:])) and np.all(out[3:] == 0)


@pytest.mark.parametrize("tree", [False, True])
def test_new_tokens_that_are_not_in_the_cache(tree):
    """kv_lens below the number of queries: the first new tokens have no key."""
    c = Case([9], [20], 4, 2, tree=tree, seed=14)
    c.kv[0] = 4
    c.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,ctx", [(12, 100), (40, 0), (70, 61), (5, 64)])
def test_nan_and_infinity_behind_the_mask(n, ctx, fp8):
    """Hidden tokens of a tree hold NaN and infinities in K and V: only the rows that see them are touched."""
    c = Case([n, 1], [ctx, 30], 4, 2, fp8, tree=True, seed=15)
    rows = c.rows(0)
    bad = [ctx + n - 1, ctx + n // 2]
    hidden = [i for i in range(n) if not any(C.sees(i, u - ctx, c.mask[i]) for u in bad)]
    ref, zref, e = c.oracle()
    k, v = c.k.view(-1, 2, 128), c.v.view(-1, 2, 128)
    nan, inf = (0x7F, 0xFF) if fp8 else (float("nan"), float("inf"))
    k[rows[bad[0]], 0, 3], v[rows[bad[0]], :, ::5] = nan, nan
    v[rows[bad[1]], 1, 7] = inf
    out, lse, st = c.gpu()
    assert st == 0 and len(hidden) > 0
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    clean = hidden + [n]
    assert np.all(np.isfinite(out[clean])) and np.all(np.isfinite(lse[:, clean]))
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * e["absav"]
    assert np.all(np.abs(out - ref)[clean] <= tol[clean])
    i = n - 1  # sees itself
    assert np.all(np.isnan(out[i][:2])) and np.all(np.isnan(out[i, 2:, ::5]))  # KV head 0: its logits are NaN
    rest = np.ones(128, dtype=bool)
    rest[::5] = False
    if not C.sees(i, bad[1] - ctx, c.mask[i]):
        assert np.all(np.isfinite(out[i, 2:][:, rest]))
    j = bad[1] - ctx
    if not C.sees(j, bad[0] - ctx, c.mask[j]):
        got = out[j, 2:, 7]
        assert np.all(np.isnan(got) if fp8 else np.isposinf(got))
        rest = np.arange(128) != 7
        assert np.all(np.abs(out - ref)[j][2:][:, rest] <= tol[j][2:][:, rest])


def test_infinity_in_a_cached_value_is_everyones():
    c = Case([3], [500], 4, 2, seed=16)
    c.v.view(-1, 2, 128)[c.rows(0)[100], 1, 9] = float("inf")
    out, _, _ = c.gpu()
    assert torch.isinf(out[:, 2:, 9]).all() and torch.isfinite(out[:, :2]).all()


def test_pages_outside_the_pool_read_zeros():
    c = Case([2], [300], 4, 2, seed=17)
    out, lse = c.check()
    c.k.view(-1, 2, 128)[c.rows(0)[64:128]] = 0
    c.v.view(-1, 2, 128)[c.rows(0)[64:128]] = 0
    want, wl, _ = c.gpu()
    for page in (-1, -2 ** 31, c.k.shape[0], 2 ** 31 - 1, 2 ** 25):
        c.table[0, 1] = page
        out, lse, st = c.gpu()
        assert st == 0 and torch.equal(out, want) and torch.equal(lse, wl)


def test_two_sequences_share_pages():
    c = Case([2, 2], [256, 256], 4, 2, seed=18)
    c.table[1, :4] = c.table[0, :4]
    c.check()


def test_values_out_of_range_are_reported():
    c = Case([2, 3, 1], [100, 50, 20], 4, 2, seed=19)
    want, wl, _ = c.gpu()
    fill = lambda: (torch.full_like(want, 7), torch.full_like(wl, 7))  # noqa: E731
    # the work is cut by all lengths, so other cuts may round otherwise: each side is within
    # 2^-8 |o| + 2^-13 sum p |v| / sum p <= 2^-8 |o| + 2^-11 of the exact value (|v| < 4 on average)
    same = lambda x, y: torch.allclose(x.float(), y.float(), rtol=2.0 ** -7, atol=2.0 ** -10)  # noqa: E731
    # a sequence whose offsets leave the batch, or go back, is skipped; the others are computed
    for cu in ([0, 2, 5, 9], [0, 2, 2 ** 31 - 1, 6], [0, 2, 1, 1], [-1, 2, 5, 6]):
        c.cu = cu
        out, lse = fill()
        out, lse, st = c.gpu(out=out, lse=lse)
        assert st == 8
        for s in range(3):
            good = 0 <= cu[s] <= cu[s + 1] <= 6
            if good and cu[s:s + 2] == [0, 2, 5, 6][s:s + 2]:
                assert same(out[cu[s]:cu[s + 1]], want[cu[s]:cu[s + 1]])
            elif not good and 0 <= cu[s] < 6:
                assert torch.all(out[cu[s]:[2, 5, 6][s]] == 7)
    c.cu = [0, 2, 5, 6]
    out, lse = fill()
    out, lse, st = c.gpu(max_seq_tokens=2, out=out, lse=lse)  # the third query of the second sequence is left out
    assert st == 8 and torch.all(out[4] == 7) and torch.all(lse[:, 4] == 7)
    keep = [0, 1, 2, 3, 5]
    assert same(out[keep], want[keep]) and same(lse[:, keep], wl[:, keep])
    c.kv[1] = -5
    out, lse, st = c.gpu()
    assert st == 8 and torch.all(out[2:5] == 0) and torch.isneginf(lse[:, 2:5]).all() and same(out[:2], want[:2])
    c.kv[1] = 10 ** 9  # past the table's row: those keys are not seen
    out, lse, st = c.gpu()
    assert st == 8 and same(out[:2], want[:2]) and same(out[5:], want[5:])


def test_rows_behind_the_last_sequence_are_left_as_they_were():
    c = Case([2, 3], [100, 50], 4, 2, seed=20, extra=4)
    out, lse = torch.full((9, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, 9), 5.0, device="cuda")
    c.check(out=out, lse=lse)
    assert torch.all(out[5:] == 5) and torch.all(lse[:, 5:] == 5)


def test_no_queries_at_all():
    c = Case([0, 0], [10, 0], 4, 2, seed=21, extra=3)
    out, lse = torch.full((3, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, 3), 5.0, device="cuda")
    out, lse, st = c.gpu(max_seq_tokens=1, out=out, lse=lse)
    assert st == 0 and torch.all(out == 5) and torch.all(lse == 5)
    c = Case([0], [10], 4, 2, seed=21)
    out, lse, st = c.gpu(max_seq_tokens=0)
    assert st == 0 and out.shape[0] == 0


def test_mask_words_that_do_not_cover_the_tokens():
    Case([50], [20], 4, 2, tree=True, words=1, seed=22).check()
    Case([5], [20], 4, 2, tree=True, words=4, seed=22).check()


def test_the_same_bits_every_time_and_on_another_stream():
    c = Case([1, 20, 3], [4000, 900, 20000], 8, 2, tree=True, seed=23)
    out, lse, _ = c.gpu()
    for _ in range(3):
        o2, l2, _ = c.gpu(max_seq_tokens=20)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, l2, _ = c.gpu(stream=s)
    s.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_captured_call_follows_growing_lengths_and_shares_its_workspace():
    """Two captured calls on one workspace, replayed while kv_lens grows."""
    c = Case([1, 1], [900, 60], 8, 2, seed=24)
    d = Case([4, 2], [300, 2000], 8, 2, seed=25, fp8=True)
    c.gpu()
    d.gpu()
    ws = torch.empty(max(b.stem_tree_ws_bytes(c.tree), b.stem_tree_ws_bytes(d.tree)), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for x in (c, d):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.stem_tree_attn(x.tree, x.cache, ws=ws)[:2])
        graphs.append(g)
    for grow in (0, 1, 3, 5):
        for x, (o, z), g in zip((c, d), outs, graphs):
            kv = x.tree.kv_lens.clone()
            x.tree.kv_lens -= grow
            g.replay()
            assert b.stem_read_device_status(ws) == 0
            o2, z2, _ = b.stem_tree_attn(x.tree, x.cache)
            assert torch.equal(o, o2) and torch.equal(z, z2)
            x.tree.kv_lens.copy_(kv)


def test_two_calls_at_once_on_their_own_workspaces():
    c = Case([30, 7], [9000, 15000], 8, 2, tree=True, seed=26)
    out, lse, _ = c.gpu()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(b.stem_tree_attn(c.tree, c.cache))
    torch.cuda.synchronize()
    for o, z, _ in got:
        assert torch.equal(o, out) and torch.equal(z, lse)


def test_pages_past_32_bit_offsets():
    P, hkv = 33000, 8
    pool = [torch.zeros(P, 64, hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    g = torch.Generator("cuda").manual_seed(1)
    pages = torch.tensor([[P - 1, 3, P - 2]], dtype=torch.int32, device="cuda")
    for p in pool:
        p[pages[0].long()] = torch.randn(3, 64, hkv, 128, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(2, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    tree = b.make_tree(q, torch.tensor([0, 2], **i32), torch.tensor([170], **i32), hkv, max_seq_tokens=2)
    out, lse, _ = b.stem_tree_attn(tree, b.paged_kv(*pool, pages, 64))
    small = [p[pages[0].long()].contiguous() for p in pool]
    o2, l2, _ = b.stem_tree_attn(tree, b.paged_kv(*small, torch.tensor([[0, 1, 2]], **i32), 64))
    assert torch.equal(out, o2) and torch.equal(lse, l2) and torch.isfinite(out.float()).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("width,over", [(1, 1000), (3, 1000), (3, 2), (4, 77), (5, 10 ** 9)])
def test_keys_past_the_tables_row_are_not_seen(width, over, n, fp8):
    """kv_lens past what the table's row holds: the queries see the keys that are there and no others."""
    c = Case([n], [width * 64 - n], 4, 2, fp8, seed=width)
    c.table, held = np.ascontiguousarray(c.table[:, :width]), width * 64
    assert c.kv == [held]
    k, v = (c.f64(x.view(-1, 2, 128)[c.rows(0)], sc) for x, sc in ((c.k, c.ks), (c.v, c.vs)))
    ctx = held + over - n
    # as the oracle's batch: the keys that every query sees, then the new tokens that are there
    fresh = max(held - ctx, 0)
    j = np.arange(n)
    mask = ((j[None, :] <= j[:, None]) & (j[None, :] < fresh)).astype(np.uint64) << (j % 32).astype(np.uint64)
    words = np.stack([mask[:, w * 32:w * 32 + 32].sum(1) for w in range(-(-n // 32))], 1).astype(np.uint32)
    seen = min(ctx, held)
    pad = lambda x: np.concatenate([x, np.zeros((n - fresh, 2, 128))])  # noqa: E731
    c.oracle = lambda: C.tree_attn(c.f64(c.q, c.qs), [pad(k)], [pad(v)], [0, n], [seen + n], words)
    c.kv[0] = held + over
    out, lse, st = c.gpu()
    assert st == 8
    got, c.kv[0], c.gpu = (out, lse, st), held, lambda: got  # bounds for the keys that exist
    c.check(status=8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("key", [10, 63, 64, 70, 99])
def test_a_nan_in_a_cached_value_is_everyones_wherever_it_lies(key, n, fp8):
    """Also in the unit of keys that the new tokens begin in, in both kernels."""
    c = Case([n], [100], 4, 2, fp8, tree=True, seed=key)
    want, wl, _ = c.gpu()
    c.v.view(-1, 2, 128)[c.rows(0)[key], 1, 9] = 0x7F if fp8 else float("nan")
    out, lse, st = c.gpu()
    assert st == 0 and torch.isnan(out[:, 2:, 9]).all()
    out[:, 2:, 9] = want[:, 2:, 9]
    assert torch.equal(out, want) and torch.equal(lse, wl)  # and nothing else is touched


@pytest.mark.parametrize("fp8", [False, True])
def test_the_largest_length(fp8):
    """2^31 - 128 keys, sixteen pages over and over: the look-ahead over the pages stays inside the table's row.
    An SM's accumulators take at most 2^31 / 148 / 16 = 2^19.8 products of 16 keys, each rounding cut off at
    2^-23; a thread's sum 2^31 / 148 / 128 = 2^16.8 weights, rounded to 2^-24."""
    P, L, hq = 16, 2 ** 31 - 128, 4
    g = torch.Generator("cuda").manual_seed(33)
    sc = [torch.full((h,), 0.01, device="cuda") for h in (hq, 1, 1)] if fp8 else [None] * 3
    x = [torch.randn(n, h, 128, generator=g, device="cuda") for n, h in ((1, hq), (P * 64, 1), (P * 64, 1))]
    enc = [(y / 0.01).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else y.to(torch.bfloat16) for y in x]
    dec = [y.view(torch.float8_e4m3fn).double() * float(s[0]) if fp8 else y.double() for y, s in zip(enc, sc)]
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(L // 64, **i32).remainder(P)[None].contiguous()
    times = torch.bincount(table[0], minlength=P).double().repeat_interleave(64)  # that each key occurs
    tree = b.make_tree(enc[0], torch.tensor([0, 1], **i32), torch.tensor([L], **i32), 1, max_seq_tokens=1,
                       q_scale=sc[0], k_scale=sc[1], v_scale=sc[2])
    out, lse, ws = b.stem_tree_attn(tree, b.paged_kv(*(y.view(P, 64, 1, 128) for y in enc[1:]), table, 64))
    assert b.stem_read_device_status(ws) == 0
    s = dec[0][0] @ dec[1][:, 0].T / 128 ** 0.5 + times.log()
    z = torch.logsumexp(s, 1)
    p = torch.exp(s - z[:, None])
    o, av = p @ dec[2][:, 0], p @ dec[2][:, 0].abs()
    assert torch.all((out[0].double() - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** (19.8 - 23) + 2.0 ** (16.8 - 24)) * av)
    assert torch.all((lse[:, 0].double() - z).abs() <= 2.0 ** (16.9 - 24))


def attention_sink(n, ctx, nats, fp8, where, ones, seed=0):
    """One key `nats` above all others, with a value of zero: the output is what the others' weights leave."""
    c = Case([n], [ctx], 4, 1, fp8, seed=seed, scale=float(nats) if nats else 1.0)
    one, rows = (0x38 if fp8 else 1.0), c.rows(0)
    if fp8:
        c.qs, c.ks, c.vs = (torch.ones(h, device="cuda") for h in (4, 1, 1))
    for x, at in ((c.q, slice(None)), (c.k.view(-1, 1, 128), rows)):
        x[at] = 0
    c.q[..., 0] = one
    v = torch.randn(len(rows), 1, 128, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")
    v = c._enc(torch.ones_like(v) if ones else v, c.vs)
    v[where] = 0
    c.v.view(-1, 1, 128)[rows] = v
    if nats:
        c.k.view(-1, 1, 128)[rows[where], 0, 0] = one
    return c


def check_tail(n, ctx, nats, fp8, where):
    """At 20 nats a weight is 2^-28.9 of the largest; in e4m3 it is off by at most 2^-9 of itself there, in bf16 by 2^-15."""
    for ones in (True, False):
        c = attention_sink(n, ctx, nats, fp8, where, ones, seed=nats)
        out, lse, st = c.gpu()
        assert st == 0
        o, z, e = c.oracle()
        out = out.double().cpu().numpy()
        logit, L = 136 * 2.0 ** -24 * e["qk"], ctx + n
        w = (2.0 ** -9 if fp8 else 2.0 ** -14) + 2 * logit + 2.0 ** -20 + 2 * L * 2.0 ** -24
        tol = 2.0 ** -8 * np.abs(o) + w[..., None] * e["absav"]
        assert np.all(np.abs(out - o) <= tol), float((np.abs(out - o) / tol).max())
        assert np.all(np.abs(lse.double().cpu().numpy() - z) <= logit.T + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * np.abs(z))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("ctx,where", [(100, 0), (8192, 0), (8192, 5000)])
@pytest.mark.parametrize("nats", [0, 6, 11, 14, 15, 16, 18, 20])
def test_the_tail_of_the_weights(nats, ctx, where, n, fp8):
    """Weights far below the largest keep their share (4 and 12 rows).  e4m3: three terms of e4m3, with the
    largest weight at 2^5 or more; below 2^-8 times 2^16, so that 2^-23.9 is off by half a step of 2^-9 2^-8 2^-16 (2^-34),
    and just above 2^-8 by 2^-18."""
    check_tail(n, ctx, nats, fp8, where)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [5, 33])
@pytest.mark.parametrize("ctx,where", [(100, 0), (8192, 0), (8192, 5000)])
@pytest.mark.parametrize("nats", [0, 6, 11, 14, 15, 16, 18, 20])
def test_the_tail_of_the_weights_in_full_tiles(nats, ctx, where, n, fp8):
    """e4m3: f16 with the largest weight at 2^13 or more, so that 2^-15.9 is off by half a step of 2^-24."""
    check_tail(n, ctx, nats, fp8, where)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [5, 40])
@pytest.mark.parametrize("scale", [1e-30, 1e-44, 1e-60])
def test_scales_below_the_range_of_fp32(scale, n, fp8):
    """All logits vanish: the mean over the keys that a query sees, and no others."""
    Case([n], [70], 4, 2, fp8, tree=True, seed=n, scale=scale).check()
    if fp8:
        c = Case([n], [70], 4, 2, fp8, tree=True, seed=n)
        c.qs, c.ks = torch.full_like(c.qs, scale ** 0.5), torch.full_like(c.ks, scale ** 0.5)
        c.check()


def test_calls_on_other_streams_use_memory_of_their_own():
    """stream=: what the call makes for itself may not be handed to a call on another stream while it is in use."""
    c = Case([30, 7], [9000, 15000], 8, 2, tree=True, seed=27)
    out, lse, _ = c.gpu()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got, places = [], {}
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(10 ** 7)  # some milliseconds: every call below is enqueued while it runs
    for s in streams * 3:
        o, z, ws = b.stem_tree_attn(c.tree, c.cache, stream=s)
        places.setdefault(ws.data_ptr(), set()).add(s)
        got.append((o, z))
        del ws
    torch.cuda.synchronize()
    assert all(len(s) == 1 for s in places.values())
    for o, z in got:
        assert torch.equal(o, out) and torch.equal(z, lse)
