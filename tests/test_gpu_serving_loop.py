"""The paged-cache operators together, as a server uses them: a prompt's step
(extend, rotate into the pages, block-sparse attention over the pages), a drafted
tree (extend with parents, rotate, tree attention), the accepted path kept, and
plain decoding after it; then the decoding step as one captured graph.  The
oracle follows with its own page tables, angles and attention."""

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C
from oracle import stem_oracle as O

pytestmark = pytest.mark.gpu

b = pytest.importorskip("block_sparse_attention_stem_b200.binding")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

HQ, HKV, PS, PAGES, MAXP = 8, 2, 64, 40, 12
FREQ = dict(scaling="yarn", factor=4.0, original_len=256, base=1e4)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Server:
    """One layer's cache and its host-side mirror (keys in fp64 by sequence)."""

    def __init__(self, S, fp8, seed):
        self.S, self.fp8, self.g = S, fp8, torch.Generator("cuda").manual_seed(seed)
        self.scales = {}
        if fp8:
            self.scales = {n + "_scale": torch.full((h,), 4.5 / 448, device="cuda") for n, h in (("q", HQ), ("k", HKV), ("v", HKV))}
        kind = torch.uint8 if fp8 else torch.bfloat16
        nan = 0x7F if fp8 else float("nan")
        self.pools = [torch.full((PAGES, PS, HKV, 128), nan, dtype=kind, device="cuda") for _ in range(2)]
        self.table = torch.full((S, MAXP), -1, dtype=torch.int32, device="cuda")
        self.cache = b.paged_kv(*self.pools, self.table, PS)
        self.held, self.cursor, self.lens = i32([0] * S), i32([0]), i32([0] * S)
        self.free = i32(np.random.default_rng(seed).permutation(PAGES))
        self.rope = b.make_rope(rotary_dim=96, layout="half", **FREQ)
        self.keys = [np.zeros((0, HKV, 128)) for _ in range(S)]
        self.vals = [np.zeros((0, HKV, 128)) for _ in range(S)]

    def project(self, T):
        x = torch.randn(T, (HQ + 2 * HKV) * 128, generator=self.g, device="cuda").to(torch.bfloat16)
        q, k, v = x.split([HQ * 128, HKV * 128, HKV * 128], dim=1)
        return q.view(T, HQ, 128), k.view(T, HKV, 128), v.view(T, HKV, 128)

    def f64(self, x, name):
        x = x.contiguous()
        if not self.fp8:
            return x.double().cpu().numpy()
        return O.e4m3_bytes_to_f64(x.view(torch.uint8).cpu().numpy()) * 4.5 / 448

    def step(self, new, parents=None, words=0):
        """extend and rotate; returns the step's maps and the rotated queries."""
        T = sum(new)
        q, k, v = self.project(T)
        st = b.stem_cache_extend(self.table, PS, PAGES, self.lens, i32(new), self.held, self.free, self.cursor, T,
                                 parents=None if parents is None else i32(parents), mask_words=words)
        q_rot, _, _ = b.stem_rope(self.rope, q, k, v, st.positions, cache=self.cache, slots=st.slots, **self.scales)
        assert b.stem_read_device_status(st.ws) == 0
        self.held, self.cursor = st.held, st.cursor
        # the oracle's own keys, from what was projected; positions counted on the host
        lens, cu = self.lens.tolist(), np.concatenate([[0], np.cumsum(new)])
        pos = []
        for s, n in enumerate(new):
            depth = {}
            for i in range(n):
                up = i - 1 if parents is None else int(parents[cu[s] + i])
                depth[i] = depth[up] + 1 if up >= 0 else 0
                pos.append(lens[s] + depth[i])
        assert st.positions.tolist() == pos
        kr, size = C.rope(k.double().cpu().numpy(), pos, 96, "half", **FREQ)
        rows = st.slots.long()
        got_k, got_v = (self.f64(p.view(-1, HKV, 128)[rows], n) for p, n in zip(self.pools, "kv"))
        want_v = v.double().cpu().numpy()
        if self.fp8:
            sc = 4.5 / 448
            lim = 448 * sc
            tol = lambda y, z: 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * sc + 2.0 ** -19 * z  # noqa: E731
            kr, want_v = np.clip(kr, -lim, lim), np.clip(want_v, -lim, lim)
            assert np.all(np.abs(got_v - want_v) <= tol(want_v, np.abs(want_v)))
        else:
            tol = lambda y, z: 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * z  # noqa: E731
            assert np.array_equal(got_v, want_v)
        assert np.all(np.abs(got_k - kr) <= tol(kr, size))
        for s, n in enumerate(new):  # attention is checked on the stored values
            self.keys[s] = np.concatenate([self.keys[s][:lens[s]], got_k[cu[s]:cu[s + 1]]])
            self.vals[s] = np.concatenate([self.vals[s][:lens[s]], got_v[cu[s]:cu[s + 1]]])
        return st, q_rot, cu

    def attend(self, st, q_rot, cu, most, mask=None):
        tree = b.make_tree(q_rot, st.cu_seqlens, st.kv_lens, HKV, mask=mask, max_seq_tokens=most, **self.scales)
        out, lse, ws = b.stem_tree_attn(tree, self.cache)
        assert b.stem_read_device_status(ws) == 0
        self.check(out, lse, q_rot, cu, None if mask is None else mask.cpu().numpy().view(np.uint32))

    def check(self, out, lse, q_rot, cu, mask=None, w=None):
        kv = [len(k) for k in self.keys]
        o, z, e = C.tree_attn(self.f64(q_rot, "q"), self.keys, self.vals, cu, kv, mask)
        logit = 136 * 2.0 ** -24 * e["qk"]
        # a weight: 2^-15 (two bf16), e4m3 2^-11 (f16, or three e4m3 terms), the sums, the logit twice
        w = w or (2.0 ** -10 if self.fp8 else 2.0 ** -14)
        tol = 2.0 ** -8 * np.abs(o) + (2 * logit + w + 2 * max(kv) * 2.0 ** -24)[..., None] * e["absav"]
        tol += (2 * max(kv) * 2.0 ** -23 * e["vmax"])[..., None] if self.fp8 else 1e-30
        assert np.all(np.abs(out.double().cpu().numpy() - o) <= tol)
        assert np.all(np.abs(lse.double().cpu().numpy() - z) <= logit.T + 2.0 ** -18 + 2.0 ** -22 * np.abs(z))


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_tree_and_decoding(fp8):
    S = 3
    sv = Server(S, fp8, 5)
    # prompts: the block-sparse kernel with every causal block listed reads the same pages
    new = [300, 64, 129]
    st, q_rot, cu = sv.step(new)
    k_all, v_all = (p.view(-1, HKV, 128)[st.slots.long()].contiguous() for p in sv.pools)
    for p in sv.pools:  # rows behind a sequence's last token, up to its last block, have to be finite there
        p.copy_(torch.where(torch.isnan(p.view(torch.float8_e4m3fn if fp8 else p.dtype).float()), torch.zeros_like(p), p))
    qkv = b.make_qkv(q_rot, k_all, v_all, cu.tolist(), **{n: sv.scales.get(n) for n in ("q_scale", "k_scale", "v_scale")})
    params = b.make_params(keep_ratio=1.0, mu=1.0)
    _, _, rp, ci, _ = b.stem_prefill(qkv, params)
    out, lse, ws = b.stem_bsa_fwd_paged(qkv, sv.cache, params, rp, ci)
    assert b.stem_read_device_status(ws) == 0
    sv.check(out, lse, q_rot, cu, w=2.0 ** -8 if not fp8 else 2.0 ** -10)  # P in one bf16 there
    sv.attend(st, q_rot, cu, max(new))  # and as a causal chunk
    sv.lens = st.kv_lens

    for accepted in ([0, 2, 5], [0]):
        # drafts: seven tokens each, two branches; then the accepted path moves to the front
        parents = np.array([-1, 0, 0, 1, 2, 2, 5] * S)
        st, q_rot, cu = sv.step([7] * S, parents, 1)
        sv.attend(st, q_rot, cu, 7, st.mask)
        rows = st.slots.long().view(S, 7)
        for p in sv.pools:
            flat = p.view(-1, HKV, 128)
            flat[rows[:, :len(accepted)]] = flat[rows[:, accepted]]
        for s in range(S):
            n = int(sv.lens[s])
            for x in (sv.keys, sv.vals):
                x[s] = np.concatenate([x[s][:n], x[s][n:][accepted]])
        sv.lens = sv.lens + len(accepted)

    for _ in range(3):
        st, q_rot, cu = sv.step([1] * S)
        sv.attend(st, q_rot, cu, 1)
        sv.lens = st.kv_lens
    assert sv.held.tolist() == [-(-max(n, 0) // PS) for n in [300 + 3 + 7, 64 + 3 + 7, 129 + 3 + 7]]  # drafts' pages are kept


def test_a_decoding_step_as_one_graph():
    """extend, rotate and attend captured once, replayed with the lengths advancing on the device."""
    S, steps = 2, 70
    sv = Server(S, False, 6)
    st, _, _ = sv.step([60, 1])
    sv.lens = st.kv_lens
    q, k, v = sv.project(S)
    e = dict(dtype=torch.int32, device="cuda")
    lens, held, cursor, new = sv.lens.clone(), sv.held.clone(), sv.cursor.clone(), i32([1] * S)
    out = b.CacheStep(held, cursor, torch.empty(S + 1, **e), lens, torch.empty(S, **e), torch.empty(S, **e), None,
                      torch.empty(256, dtype=torch.uint8, device="cuda"))
    q_rot = torch.empty(S, HQ, 128, dtype=torch.bfloat16, device="cuda")
    tree = b.make_tree(q_rot, out.cu_seqlens, lens, HKV, max_seq_tokens=1)
    ws = torch.empty(b.stem_tree_ws_bytes(tree), dtype=torch.uint8, device="cuda")
    o, z = torch.empty(S, HQ, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(HQ, S, device="cuda")

    def step():
        b.stem_cache_extend(sv.table, PS, PAGES, lens, new, held, sv.free, cursor, S, out=out)
        b.stem_rope(sv.rope, q, k, v, out.positions, cache=sv.cache, slots=out.slots, q_out=q_rot)
        b.stem_tree_attn(tree, sv.cache, out=o, lse=z, ws=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps):
        g = torch.randn(k.shape, generator=sv.g, device="cuda").to(torch.bfloat16)
        k.copy_(g)
        v.copy_(-g)
        q.copy_(torch.randn(q.shape, generator=sv.g, device="cuda").to(torch.bfloat16))
        graph.replay()
        rows = out.slots.long()
        for s in range(S):
            for x, p in ((sv.keys, 0), (sv.vals, 1)):
                x[s] = np.concatenate([x[s], sv.f64(sv.pools[p].view(-1, HKV, 128)[rows[s:s + 1]], "k")])
        assert lens.tolist() == [len(x) for x in sv.keys]
        sv.check(o, z, q_rot, np.array([0, 1, 2]))
    assert b.stem_read_device_status(ws) == 0 and b.stem_read_device_status(out.ws) == 0
    assert held.tolist() == [3, 2] and int(cursor) == 5


def test_outputs_of_calls_on_another_stream_belong_to_it():
    """Memory that a call made on `stream` is not handed to the current stream when it is dropped."""
    T, S = 300, 2
    g = torch.Generator("cuda").manual_seed(7)
    q, k, v = (torch.randn(T, h, 128, generator=g, device="cuda").to(torch.bfloat16) for h in (HQ, HKV, HKV))
    qkv, params = b.make_qkv(q, k, v, [0, 130, T]), b.make_params()
    scores, _, _ = b.stem_score(qkv, params)
    _, rp, ci, _ = b.stem_select(qkv, params, scores)
    pages = [torch.zeros(8, PS, HKV, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache = b.paged_kv(*pages, i32([[0, 1, 2, -1], [3, 4, 5, -1]]), PS)
    tree = b.make_tree(q, i32([0, 130, T]), i32([130, T - 130]), HKV)
    pos, table = i32(np.arange(T)), i32(np.full((S, 8), -1))
    step = [i32(x) for x in ([0, 5], [3, 4], [0, 1], [6, 7, 8], [0])]
    calls = [
        lambda **kw: b.stem_score(qkv, params, **kw),
        lambda **kw: b.stem_select(qkv, params, scores, **kw),
        lambda **kw: b.stem_score_select(qkv, params, **kw),
        lambda **kw: b.stem_bsa_fwd(qkv, params, rp, ci, **kw),
        lambda **kw: b.stem_bsa_fwd_paged(qkv, cache, params, rp, ci, **kw),
        lambda **kw: b.stem_prefill(qkv, params, **kw),
        lambda **kw: b.stem_rope(b.make_rope(), q, k, v, pos, **kw),
        lambda **kw: b.stem_tree_attn(tree, cache, **kw),
        lambda **kw: vars(b.stem_cache_extend(table, PS, 64, *step, 9, **kw)).values(),
    ]
    for call in calls:
        s = torch.cuda.Stream()
        want = [t for t in call() if t is not None]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(10 ** 7)
        got = [t for t in call(stream=s) if t is not None]
        shapes = [(t.shape, t.dtype) for t in got]
        places = {t.untyped_storage().data_ptr() for t in got if t.numel()}
        s.synchronize()
        # (the workspace, whose scratch is nobody's, is the last one)
        assert all(torch.equal(x, y) for x, y in zip(want[:-1], got[:-1]))
        del got
        fresh = [torch.empty(shape, dtype=dt, device="cuda") for shape, dt in shapes for _ in range(2)]
        assert places.isdisjoint(t.untyped_storage().data_ptr() for t in fresh)
        del fresh
