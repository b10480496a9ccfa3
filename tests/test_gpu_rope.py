"""stem_rope on the GPU against the fp64 oracle.

Bounds, relative to s = amplitude (|a| + |b|) of the pair: the angle is off by at
most 2^-25 half turns from the fp32 conversion (9.4e-8 rad) and 2^-31 from the
dropped bits, sincospif by 2 ulp (2^-23), the amplitude, two products and the sum
by 2^-24 each: together below 7e-7 < 2^-20 s.  Outputs round once more: half a step
(bf16 2^-8, e4m3 2^-4 relative or 2^-10 absolute below its normal range).  The
scaling by the fp32 reciprocal of the scale adds 2^-23."""

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C
from oracle import stem_oracle as O

pytestmark = pytest.mark.gpu

b = pytest.importorskip("block_sparse_attention_stem_b200.binding")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def f64(x):
    return x.detach().double().cpu().numpy()


def values(x):
    """fp64 values of a bf16 tensor or of e4m3 bytes."""
    return O.e4m3_bytes_to_f64(x.view(torch.uint8).cpu().numpy()) if x.element_size() == 1 else f64(x)


def bound(y, size, fp8):
    return (2.0 ** -4 * np.abs(y) + 2.0 ** -10 + 2.0 ** -19 * size) if fp8 else (2.0 ** -8 * np.abs(y) + 2.0 ** -20 * size)


def make(T, hq, hkv, seed, fused=True):
    g = torch.Generator("cuda").manual_seed(seed)
    n = (hq + 2 * hkv) * 128
    x = torch.randn(T, n + (64 if fused else 0), generator=g, device="cuda", dtype=torch.bfloat16)[:, :n]  # padded rows
    q, k, v = x.split([hq * 128, hkv * 128, hkv * 128], dim=1)
    return q.view(T, hq, 128), k.view(T, hkv, 128), v.view(T, hkv, 128)


def scales(h, seed):
    return torch.rand(h, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * 0.02 + 0.002


FREQ = [dict(), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0, base=1e4),
        dict(scaling="yarn", factor=4.0, original_len=32768), dict(scaling="yarn", factor=1.0, original_len=1),
        dict(amplitude=0.5)]


def check(T, hq, hkv, rotary, layout, freq, fp8, first=0, pages=None, seed=0):
    q, k, v = make(T, hq, hkv, seed)
    pos = (torch.arange(T, dtype=torch.int64) * 37 + first).to(torch.int32)
    kw = {}
    if fp8:
        kw = dict(q_scale=scales(hq, 1), k_scale=scales(hkv, 2), v_scale=scales(hkv, 3))
    rope = b.make_rope(rotary_dim=rotary, layout=layout, **freq)
    cache = slots = before = None
    if pages:
        ps, P = pages
        kind = torch.uint8 if fp8 else torch.bfloat16
        pool = [torch.full((P, ps, hkv, 128), 3, dtype=kind, device="cuda") for _ in range(2)]
        slots = torch.from_numpy(np.random.default_rng(seed).permutation(P * ps)[:T].astype(np.int32)).cuda()
        if T > 4:
            slots[2], slots[4] = -1, P * ps + 3  # tokens that are not stored
        cache = b.paged_kv(*pool, torch.zeros(1, P, dtype=torch.int32, device="cuda"), ps)
        before = [p.clone() for p in pool]
    qo, ko, vo = b.stem_rope(rope, q, k, v, pos.cuda(), cache=cache, slots=slots, **kw)
    torch.cuda.synchronize()

    def expect(x, sc, turn=True):
        y, size = C.rope(f64(x), pos.numpy(), rotary, layout, **freq) if turn else (f64(x), np.abs(f64(x)))
        if fp8:
            s = f64(sc)[None, :, None]
            y, size = np.clip(y / s, -448, 448), size / s
        return y, size

    qy, qs = expect(q, kw.get("q_scale"))
    ky, ks = expect(k, kw.get("k_scale"))
    vy, vs = expect(v, kw.get("v_scale"), turn=False)
    assert np.all(np.abs(values(qo) - qy) <= bound(qy, qs, fp8))
    if pages:
        assert ko is None and vo is None
        at = slots.cpu().numpy()
        kept = (at >= 0) & (at < pages[0] * pages[1])
        rows = [p.view(-1, hkv, 128) for p in pool]
        ko, vo = (r[slots[torch.from_numpy(kept).cuda()].long()] for r in rows)
        for r, old in zip(rows, before):
            untouched = np.ones(len(r), dtype=bool)
            untouched[at[kept]] = False
            u = torch.from_numpy(untouched).cuda()
            assert torch.equal(r[u], old.view(-1, hkv, 128)[u])
        ky, ks, vy, vs = ky[kept], ks[kept], vy[kept], vs[kept]
    assert np.all(np.abs(values(ko) - ky) <= bound(ky, ks, fp8))
    if fp8:
        assert np.all(np.abs(values(vo) - vy) <= bound(vy, vs, True))
    else:
        assert np.array_equal(values(vo), vy)  # v is only stored
        if rotary < 128:  # and so is the part of a head that is not rotated
            assert torch.equal(qo[..., rotary:], q[..., rotary:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rotary", [16, 48, 64, 96, 112, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_layouts_and_parts_of_the_head(layout, rotary, fp8):
    check(67, 6, 2, rotary, layout, dict(), fp8, first=1000)


@pytest.mark.parametrize("freq", FREQ)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_scalings(freq, layout):
    check(40, 4, 2, 128, layout, freq, False, first=90000)


@pytest.mark.parametrize("first", [0, -500, 2 ** 20, 2 ** 31 - 200, -2 ** 31])
def test_far_positions(first):
    check(5, 2, 1, 128, "half", dict(base=10.0), False, first=first)


@pytest.mark.parametrize("T,hq,hkv", [(1, 32, 8), (1, 1, 1), (2, 5, 5), (7, 3, 1), (8, 64, 8), (9, 12, 4), (300, 40, 8),
                                      (2500, 32, 8)])
@pytest.mark.parametrize("fp8", [False, True])
def test_pages(T, hq, hkv, fp8):
    check(T, hq, hkv, 128, "half", dict(), fp8, first=3, pages=(64, T // 64 + 2), seed=T)


@pytest.mark.parametrize("ps", [64, 192])
def test_pages_of_other_sizes(ps):
    check(500, 8, 2, 64, "interleaved", dict(), False, pages=(ps, 500 // ps + 2))


def test_in_place_and_single_tensors():
    q, k, v = (x.contiguous() for x in make(33, 4, 2, 9))
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    rope = b.make_rope()
    q1, k1, v1 = b.stem_rope(rope, q, k, v, pos)
    q2, none_k, none_v = b.stem_rope(rope, q, None, None, pos)
    assert none_k is None and none_v is None and torch.equal(q1, q2)
    none_q, k2, _ = b.stem_rope(rope, None, k, None, pos)
    assert none_q is None and torch.equal(k1, k2) and torch.equal(v1, v)
    _, _, v2 = b.stem_rope(rope, None, None, v, pos)
    assert torch.equal(v2, v)
    b.stem_rope(rope, q, k, v, pos, q_out=q, k_out=k)
    assert torch.equal(q, q1) and torch.equal(k, k1)


def test_no_tokens():
    q, k, v = make(4, 2, 1, 3)
    qo, ko, vo = b.stem_rope(b.make_rope(), q[:0], k[:0], v[:0], torch.empty(0, dtype=torch.int32, device="cuda"))
    assert qo.shape == (0, 2, 128) and ko.shape == vo.shape == (0, 1, 128)


def test_rotating_back_gives_the_input():
    q, k, v = make(50, 2, 2, 4)
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 1001
    rope = b.make_rope()
    q1, _, _ = b.stem_rope(rope, q, None, None, pos)
    q2, _, _ = b.stem_rope(rope, q1, None, None, -pos)
    # two roundings to bf16 of a pair whose length is kept, each 2^-8 of an element of at most that length
    size = C.rope(f64(q), np.zeros(50), 128, "half")[1]
    assert np.all(np.abs(f64(q2) - f64(q)) <= (2 * 2.0 ** -8 * 1.5 + 2.0 ** -18) * size)


@pytest.mark.parametrize("fp8", [False, True])
def test_nan_and_infinity_stay_in_their_pair(fp8):
    q, k, v = (x.clone() for x in make(3, 2, 2, 5))
    q[1, 0, 5], k[2, 1, 70], v[0, 0, 3], v[1, 1, 9] = float("nan"), float("inf"), float("nan"), float("-inf")
    kw = dict(q_scale=scales(2, 1), k_scale=scales(2, 2), v_scale=scales(2, 3)) if fp8 else {}
    pos = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    qo, ko, vo = (values(x) for x in b.stem_rope(b.make_rope(), q, k, v, pos, **kw))
    bad = np.argwhere(~np.isfinite(qo)).tolist()
    assert bad == [[1, 0, 5], [1, 0, 69]]
    odd = ~np.isfinite(ko) | (np.abs(ko) == 448) if fp8 else ~np.isfinite(ko)
    assert {tuple(x) for x in np.argwhere(odd)} >= {(2, 1, 70), (2, 1, 6)}
    assert np.isnan(vo[0, 0, 3]) and vo[1, 1, 9] == (-448 if fp8 else -np.inf)


def test_rows_past_32_bit_offsets():
    P, hkv = 33000, 8  # 33000 * 64 * 8 * 128 elements: byte offsets past 2^32
    pool = [torch.zeros(P, 64, hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q, k, v = make(3, 8, hkv, 6)
    slots = torch.tensor([5, P * 64 - 1, P * 64 - 70], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    cache = b.paged_kv(*pool, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 64)
    _, k1, v1 = b.stem_rope(b.make_rope(), q, k, v, pos)
    b.stem_rope(b.make_rope(), q, k, v, pos, cache=cache, slots=slots)
    for p, x in zip(pool, (k1, v1)):
        rows = p.view(-1, hkv, 128)
        assert torch.equal(rows[slots.long()], x)
        assert int(torch.count_nonzero(rows.view(-1, 1024).any(1))) == 3


@pytest.mark.parametrize("freq,same", [
    (dict(factor=4.0, original_len=4, base=1e4), dict(scaling="linear", factor=4.0, base=1e4)),  # all pairs too slow
    (dict(factor=8.0, original_len=1), dict(scaling="linear", factor=8.0)),
    (dict(factor=4.0, original_len=32768, base=10.0), dict(base=10.0))])  # all pairs fast enough
def test_yarn_whose_ramp_lies_outside_the_pairs(freq, same):
    """Then every pair is interpolated, or none."""
    q, k, v = make(40, 4, 2, 11)
    pos = torch.arange(40, dtype=torch.int32, device="cuda") + 90000
    one = dict(amplitude=1.0)
    q1, k1, _ = b.stem_rope(b.make_rope(scaling="yarn", **freq, **one), q, k, v, pos)
    q2, k2, _ = b.stem_rope(b.make_rope(**same, **one), q, k, v, pos)
    assert torch.equal(q1, q2) and torch.equal(k1, k2)


def test_ntk_whose_base_passes_a_double():
    """The enlarged base is about 10^320: the same angles as with the base that it is (log-space, position 1 to 40)."""
    q, k, v = make(40, 4, 2, 12)
    pos = torch.arange(1, 41, dtype=torch.int32, device="cuda")
    base, factor = 1e300, 1e20
    qo, _, _ = b.stem_rope(b.make_rope(scaling="ntk", base=base, factor=factor), q, k, v, pos)
    ln = np.log(base) + 128 / 126 * np.log(factor)
    ang = f64(pos)[:, None, None] * np.exp(-2.0 * np.arange(64) / 128 * ln)
    x, y = f64(q)[..., :64], f64(q)[..., 64:]
    want = np.concatenate([x * np.cos(ang) - y * np.sin(ang), y * np.cos(ang) + x * np.sin(ang)], -1)
    size = np.tile(np.abs(x) + np.abs(y), 2)
    assert np.all(np.abs(f64(qo) - want) <= bound(want, size, False))
