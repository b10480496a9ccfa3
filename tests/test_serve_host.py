"""Host-side checks of the paged-cache operators (no GPU needed, no kernel is
launched): refusals of the C entry points and of the binding, workspace sizes,
and the fp64 oracle's own pins."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C

b = pytest.importorskip("block_sparse_attention_stem_b200.binding")

FAKE = 1 << 20  # never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED, SMALL, MISALIGNED = range(5)


def step(**kw):
    base = dict(num_seqs=2, max_tokens=8, page_size=64, num_pages=16, max_pages_per_seq=4, num_free=4, mask_words=0,
                cache_lens=FAKE, new_lens=FAKE, held_pages=FAKE, free_pages=FAKE, cursor=FAKE, parents=None)
    base.update(kw)
    return b.StemCacheStep(*[base[f] for f, _ in b.StemCacheStep._fields_])


def extend(desc, mask=None, ws_bytes=256, **null):
    out = [None if null.get(n) else FAKE
           for n in ("table", "held", "cursor", "cu", "kv", "slots", "positions")]
    return b.LIB.stem_cache_extend(ctypes.byref(desc), *out, mask, None if null.get("ws") else FAKE, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), INVALID), (dict(num_seqs=8193), UNSUPPORTED), (dict(max_tokens=-1), INVALID),
    (dict(page_size=0), INVALID), (dict(page_size=96), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_pages=1 << 25), INVALID), (dict(max_pages_per_seq=0), INVALID),
    (dict(num_seqs=4096, max_pages_per_seq=1 << 20), INVALID), (dict(max_tokens=(1 << 30) + 1), INVALID),
    (dict(num_seqs=2, max_pages_per_seq=(1 << 29) + 1), INVALID), (dict(num_free=-1), INVALID),
    (dict(cache_lens=None), INVALID), (dict(new_lens=None), INVALID), (dict(held_pages=None), INVALID),
    (dict(cursor=None), INVALID), (dict(free_pages=None), INVALID),
    (dict(parents=FAKE, mask_words=1), INVALID),  # parents without a mask
])
def test_extend_refuses(kw, code):
    assert extend(step(**kw)) == code


def test_extend_refuses_missing_outputs():
    for n in ("table", "held", "cursor", "cu", "kv", "slots", "positions", "ws"):
        assert extend(step(), **{n: True}) == INVALID
    assert extend(step(), ws_bytes=255) == SMALL
    assert extend(step(), mask=FAKE) == INVALID                              # a mask without parents
    assert extend(step(parents=FAKE, mask_words=0), mask=FAKE) == INVALID


def rope_call(rope=None, cache=None, **kw):
    base = dict(num_tokens=4, num_q_heads=4, num_kv_heads=2, head_dim=128, out_dtype=0, positions=FAKE, slots=FAKE,
                q=FAKE, k=FAKE, v=FAKE, q_stride=512, k_stride=256, v_stride=256, q_scale=None, k_scale=None,
                v_scale=None, q_out=2 * FAKE, k_out=2 * FAKE, v_out=2 * FAKE)
    base.update(kw)
    io = b.StemRopeIO(*[base[f] for f, _ in b.StemRopeIO._fields_])
    return b.LIB.stem_rope(ctypes.byref(rope or b.make_rope()), ctypes.byref(io),
                           None if cache is None else ctypes.byref(cache), None)


@pytest.mark.parametrize("kw,code", [
    (dict(rotary_dim=0), INVALID), (dict(rotary_dim=130), INVALID), (dict(rotary_dim=33), INVALID),
    (dict(rotary_dim=24), UNSUPPORTED), (dict(base=1.0), INVALID), (dict(base=math.inf), INVALID),
    (dict(scaling="linear", factor=0.5), INVALID), (dict(scaling="ntk", factor=math.nan), INVALID),
    (dict(scaling="yarn", factor=4.0, original_len=0), INVALID), (dict(scaling="yarn", factor=4.0, beta_slow=0.0), INVALID),
    (dict(scaling="yarn", factor=4.0, beta_fast=1.0, beta_slow=2.0), INVALID), (dict(amplitude=-1.0), INVALID),
])
def test_rope_refuses_parameters(kw, code):
    assert rope_call(b.make_rope(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), INVALID), (dict(num_q_heads=-1), INVALID), (dict(head_dim=64), UNSUPPORTED),
    (dict(head_dim=0), INVALID), (dict(out_dtype=2), INVALID), (dict(positions=None), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(q_stride=504), INVALID), (dict(q_stride=516), INVALID), (dict(k_stride=1 << 62), INVALID),
    (dict(q=FAKE + 8), MISALIGNED), (dict(k_out=2 * FAKE + 8), MISALIGNED),
    (dict(out_dtype=1), INVALID),                                  # e4m3 without scales
    (dict(q_out=FAKE, q_stride=1024), INVALID),                    # in place, but not packed
    (dict(v_out=FAKE), INVALID),                                   # v is never rotated in place
    (dict(q_out=None, k_out=None, v_out=None), INVALID),           # nothing to do
])
def test_rope_refuses_tensors(kw, code):
    assert rope_call(**kw) == code


def test_rope_refuses_caches():
    pool = lambda **kw: b.StemPagedKV(*[dict(dict(page_size=64, num_pages=4, max_pages_per_seq=1, page_table=None,  # noqa: E731
                                                  k_pages=FAKE, v_pages=FAKE), **kw)[f] for f, _ in b.StemPagedKV._fields_])
    assert rope_call(cache=pool(page_size=32)) == INVALID
    assert rope_call(cache=pool(num_pages=0)) == INVALID
    assert rope_call(cache=pool(k_pages=None)) == INVALID
    assert rope_call(cache=pool(v_pages=FAKE + 4)) == MISALIGNED
    assert rope_call(cache=pool(), slots=None) == INVALID
    assert rope_call(cache=pool(), num_tokens=0) == OK  # nothing to do, nothing launched


def tree(**kw):
    base = dict(dtype=0, num_seqs=2, total_tokens=8, max_seq_tokens=4, num_q_heads=8, num_kv_heads=2, head_dim=128,
                mask_words=0, cu_seqlens=FAKE, kv_lens=FAKE, mask=None, q=FAKE, q_scale=None, k_scale=None, v_scale=None,
                softmax_scale=0.0)
    base.update(kw)
    return b.StemTree(*[base[f] for f, _ in b.StemTree._fields_])


def plan(desc):
    n = ctypes.c_size_t(0)
    return b.LIB.stem_tree_plan(ctypes.byref(desc), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), INVALID), (dict(num_seqs=0), INVALID), (dict(total_tokens=-1), INVALID),
    (dict(max_seq_tokens=-1), INVALID), (dict(num_q_heads=7), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(num_q_heads=129, num_kv_heads=1), UNSUPPORTED), (dict(head_dim=64), UNSUPPORTED), (dict(head_dim=0), INVALID),
    (dict(total_tokens=(1 << 30) + 1), UNSUPPORTED), (dict(num_seqs=1 << 30), UNSUPPORTED),
    (dict(mask=FAKE, mask_words=0), INVALID), (dict(softmax_scale=-1.0), INVALID), (dict(softmax_scale=math.nan), INVALID),
])
def test_tree_plan_refuses(kw, code):
    assert plan(tree(**kw))[0] == code


def test_tree_workspace_never_shrinks_with_the_lengths():
    for hq, hkv in ((1, 1), (8, 2), (12, 4), (128, 1)):
        last = 0
        for T in (0, 1, 2, 31, 32, 33, 64, 127, 128, 129, 1000, 5000, 40000):
            st, n = plan(tree(total_tokens=T, max_seq_tokens=0, num_q_heads=hq, num_kv_heads=hkv))
            assert st == OK and n >= last and n < 1 << 28
            last = n
        assert plan(tree(total_tokens=64, max_seq_tokens=1, num_q_heads=hq, num_kv_heads=hkv))[1] <= last


@pytest.mark.parametrize("kw,pool,code", [
    (dict(), dict(page_size=96), INVALID), (dict(), dict(num_pages=0), INVALID), (dict(), dict(max_pages_per_seq=0), INVALID),
    (dict(), dict(page_table=None), INVALID), (dict(), dict(k_pages=None), INVALID), (dict(), dict(v_pages=FAKE + 8), MISALIGNED),
    (dict(q=None), dict(), INVALID), (dict(q=FAKE + 2), dict(), MISALIGNED), (dict(cu_seqlens=None), dict(), INVALID),
    (dict(kv_lens=None), dict(), INVALID), (dict(dtype=1), dict(), INVALID),
])
def test_tree_attn_refuses(kw, pool, code):
    base = dict(page_size=64, num_pages=4, max_pages_per_seq=2, page_table=FAKE, k_pages=FAKE, v_pages=FAKE)
    base.update(pool)
    kv = b.StemPagedKV(*[base[f] for f, _ in b.StemPagedKV._fields_])
    assert b.LIB.stem_tree_attn(ctypes.byref(tree(**kw)), ctypes.byref(kv), FAKE, FAKE, FAKE, 1 << 40, None) == code


def test_tree_attn_refuses_a_small_workspace():
    kv = b.StemPagedKV(64, 4, 2, FAKE, FAKE, FAKE)
    n = plan(tree())[1]
    assert b.LIB.stem_tree_attn(ctypes.byref(tree()), ctypes.byref(kv), FAKE, FAKE, FAKE, n - 1, None) == SMALL
    assert b.LIB.stem_tree_attn(ctypes.byref(tree()), ctypes.byref(kv), FAKE, FAKE, None, n, None) == INVALID
    assert b.LIB.stem_tree_attn(ctypes.byref(tree()), None, FAKE, FAKE, FAKE, n, None) == INVALID


def test_binding_refuses_wrong_tensors():
    i32 = torch.int32
    table, one, cur = torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32)
    args = dict(cache_lens=one, new_lens=one, held_pages=one, free_pages=torch.zeros(8, dtype=i32), cursor=cur, max_tokens=4)

    def ext(**kw):
        return lambda: b.stem_cache_extend(kw.pop("table", table), 64, 16, **{**args, **kw})

    for bad in (ext(cache_lens=one.long()), ext(new_lens=torch.zeros(3, dtype=i32)), ext(table=table.t()),
                ext(cursor=torch.zeros(2, dtype=i32)), ext(parents=torch.zeros(5, dtype=i32), mask_words=1)):
        with pytest.raises(ValueError):
            bad()

    bf = torch.bfloat16
    q, k = torch.zeros(4, 4, 128, dtype=bf), torch.zeros(4, 2, 128, dtype=bf)
    pos = torch.zeros(4, dtype=i32)
    rope = b.make_rope()
    pages = torch.zeros(2, 64, 2, 128, dtype=bf)
    cache = b.paged_kv(pages, pages.clone(), torch.zeros(1, 2, dtype=i32), 64)
    for bad in (lambda: b.stem_rope(rope, q.float(), k, k, pos), lambda: b.stem_rope(rope, q[:3], k, k, pos),
                lambda: b.stem_rope(rope, q.transpose(0, 1), k, k, pos), lambda: b.stem_rope(rope, q, k, k, pos.long()),
                lambda: b.stem_rope(rope, q, k, q, pos), lambda: b.stem_rope(rope, q, k, k, pos, cache=cache),
                lambda: b.stem_rope(rope, q, k, None, pos, cache=cache, slots=pos),
                lambda: b.stem_rope(rope, q, q, q, pos, cache=cache, slots=pos),       # other heads than the pages
                lambda: b.stem_rope(rope, q, k, k, pos, cache=cache, slots=pos, k_scale=torch.ones(2)),  # bf16 pages
                lambda: b.stem_rope(rope, q, k, k, pos, q_out=torch.zeros(4, 4, 128)),
                lambda: b.stem_rope(rope, q, k, k, pos, q_scale=torch.ones(3))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(KeyError):
        b.make_rope(layout="pairs")

    cu, kv = torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32)
    t = b.make_tree(q, cu, kv, 2)
    for bad in (lambda: b.make_tree(q.float(), cu, kv, 2), lambda: b.make_tree(q, cu.long(), kv, 2),
                lambda: b.make_tree(q, torch.zeros(3, dtype=i32), kv, 2),
                lambda: b.make_tree(q, cu, kv, 2, mask=torch.zeros(3, 1, dtype=i32)),
                lambda: b.make_tree(q.view(torch.uint8)[..., :128].contiguous(), cu, kv, 2),  # e4m3 without scales
                lambda: b.stem_tree_attn(t, b.paged_kv(pages.view(torch.uint8), pages.view(torch.uint8), cache.page_table, 64)),
                lambda: b.stem_tree_attn(t, cache, out=torch.zeros(4, 4, 128)),
                lambda: b.stem_tree_attn(t, cache, lse=torch.zeros(4, 4, dtype=bf)),
                lambda: b.stem_tree_attn(b.make_tree(q, torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), 2), cache)):
        with pytest.raises(ValueError):
            bad()


def test_status_strings_of_the_device_errors():
    assert "out of range" in b.stem_status_string(8) and "pages" in b.stem_status_string(9)
    assert b.STATUS_NAMES[8] == "STEM_ERR_BAD_INPUT" and b.STATUS_NAMES[9] == "STEM_ERR_OUT_OF_PAGES"


# ------------------------------------------------------------------ the oracle's pins
def test_oracle_rope_keeps_lengths_and_relative_positions():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 128))
    for layout in ("half", "interleaved"):
        dots = []
        for p0 in (0, 5, 100000):
            a, _ = C.rope(q, [p0 + 7], 128, layout)
            c, _ = C.rope(k, [p0], 128, layout)
            assert np.linalg.norm(a) == pytest.approx(np.linalg.norm(q), rel=1e-12)
            dots.append(float((a * c).sum()))
        assert np.allclose(dots, dots[0], atol=1e-7)  # only the distance matters
    y, _ = C.rope(q, [9], 48, "half")
    assert np.array_equal(y[..., 48:], q[..., 48:])


def test_oracle_rope_scalings():
    w, a = C.rope_frequencies(128, scaling="plain")
    assert w[0] == 1.0 and a == 1.0
    assert np.allclose(C.rope_frequencies(128, scaling="linear", factor=4.0)[0], w / 4)
    ntk = C.rope_frequencies(128, scaling="ntk", factor=4.0)[0]
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(w[-1] / 4)  # the slowest pair is interpolated exactly
    y, a = C.rope_frequencies(128, scaling="yarn", factor=4.0, original_len=32768)
    assert y[0] == w[0] and y[-1] == pytest.approx(w[-1] / 4) and a == pytest.approx(0.1 * math.log(4) + 1)
    assert np.all(np.diff(y) < 0)


def test_oracle_tree_of_a_chain_is_causal_attention():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((3, 2, 16))
    k, v = rng.standard_normal((2, 7, 1, 16))
    chain = np.array([[1], [3], [7]], dtype=np.uint32)
    o1, l1, _ = C.tree_attn(q, [k], [v], [0, 3], [7], chain)
    o2, l2, _ = C.tree_attn(q, [k], [v], [0, 3], [7])
    assert np.array_equal(o1, o2) and np.array_equal(l1, l2)
    x = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), torch.from_numpy(k).transpose(0, 1).expand(2, -1, -1),
        torch.from_numpy(v).transpose(0, 1).expand(2, -1, -1),
        attn_mask=torch.ones(3, 7, dtype=torch.bool).tril(4)).transpose(0, 1).numpy()
    assert np.allclose(o1, x, atol=1e-12)


def test_oracle_extend_of_a_small_step():
    r = C.extend([[5, -1], [6, 7]], 64, 10, [63, 64], [2, 1], [1, 2], [9, 8], 0, 5)
    assert r["table"].tolist() == [[5, 9], [6, 7]] and r["held"].tolist() == [2, 2] and r["cursor"] == 1
    assert r["slots"].tolist() == [5 * 64 + 63, 9 * 64, 7 * 64, -1, -1] and r["positions"].tolist() == [63, 64, 64, 0, 0]
    assert r["cu"].tolist() == [0, 2, 3] and r["kv"].tolist() == [65, 65] and not r["status"]
    t = C.extend([[0, -1]], 64, 10, [3], [4], [1], [], 0, 4, parents=[-1, 0, 0, 1], mask_words=1)
    assert t["mask"][:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011] and t["positions"].tolist() == [3, 4, 4, 5]


@pytest.mark.parametrize("scale,code", [(1e-300, OK), (2.0 ** 127, OK), (2.0 ** 127 * 1.001, INVALID), (1e300, INVALID),
                                        (math.inf, INVALID)])
def test_tree_plan_refuses_scales_past_fp32(scale, code):
    assert plan(tree(softmax_scale=scale))[0] == code


def test_binding_refuses_workspaces_that_are_elsewhere_or_have_gaps():
    i32 = torch.int32
    pages = torch.zeros(2, 64, 2, 128, dtype=torch.bfloat16)
    table = torch.zeros(2, 2, dtype=i32)
    t = b.make_tree(torch.zeros(4, 4, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), 2)
    n = b.stem_tree_ws_bytes(t)
    two = torch.zeros(2, dtype=i32)
    for ws in (torch.empty(n, dtype=torch.uint8, device="meta"), torch.empty(1, dtype=torch.uint8).expand(n),
               torch.empty(2 * n, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="ws must be"):
            b.stem_tree_attn(t, b.paged_kv(pages, pages.clone(), table, 64), ws=ws)
        with pytest.raises(ValueError, match="ws must be"):
            b.stem_cache_extend(table, 64, 16, two, two, two, torch.zeros(8, dtype=i32), torch.zeros(1, dtype=i32), 4, ws=ws)


def test_oracle_yarn_outside_the_pairs():
    w = lambda **kw: C.rope_frequencies(128, **kw)[0]  # noqa: E731
    assert np.allclose(w(scaling="yarn", factor=4.0, original_len=4, base=1e4), w(base=1e4) / 4, rtol=1e-15)
    assert np.allclose(w(scaling="yarn", factor=4.0, original_len=32768, base=10.0), w(base=10.0), rtol=1e-15)
    for n in (1, 4, 7, 40, 256, 32768):  # faster pairs are never interpolated more than slower ones
        assert np.all(np.diff(w(scaling="yarn", factor=4.0, original_len=n, base=1e4) / w(base=1e4)) <= 1e-15)
