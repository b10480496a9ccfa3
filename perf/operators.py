"""Cases of the paged-cache operators: `stem_cache_extend` (page tables, slot
maps and tree masks from request lengths), `stem_rope` (rotary positions, with
K and V written into the pages) and `stem_tree_attn` (attention of drafted
trees, single tokens or causal chunks over the paged cache).

`own` selects the framework's kernels; otherwise `run` is the plain form in
elementary torch operations, in fp32 (angles in fp64), rounded once at the end.
"""

import math

import numpy as np
import torch

own = False

HEAD = 128


# ------------------------------------------------------------------ the cases
def _extend(name, **kw):
    return dict(op="extend", name=name, **kw)


def _rope(name, **kw):
    base = dict(hq=32, hkv=8, rotary=128, layout="half", scaling="plain", factor=1.0, fp8=False, page=64, pos=4096)
    base.update(kw)
    return dict(op="rope", name=name, **base)


def _attn(name, **kw):
    base = dict(hq=32, hkv=8, fp8=False, page=64, tree=False)
    base.update(kw)
    return dict(op="attn", name=name, **base)


def listed():
    return [
        # a few requests, one new token each: the step before every layer stack of a small server
        _extend("extend_tokens", seqs=4, new_lo=1, new_hi=1, cache_hi=2048, page=64, tree=False),
        # a full batch of speculative requests, drafted trees of different sizes
        _extend("extend_trees", seqs=256, new_lo=17, new_hi=64, cache_hi=32768, page=64, tree=True),
        # packed prefill of long prompts (the lengths' order of the fp8 varlen stack)
        _extend("extend_prompts", seqs=4, new_lo=8192, new_hi=98304, cache_hi=0, page=128, tree=False),
        # one decoded token of one request
        _rope("rope_token", tokens=1, pos=131072),
        # one prefill chunk (odd length), rotary part of the head, interleaved pairs, interpolated positions
        _rope("rope_chunk", tokens=2047, rotary=64, layout="interleaved", scaling="linear", factor=8.0, pos=32768),
        # the 32K prefill layer, positions past the trained length
        _rope("rope_prompt", tokens=32768, scaling="yarn", factor=4.0, pos=131072),
        # the e4m3 layer: quantised q and pages, whole long prompt
        _rope("rope_prompt_fp8", tokens=98304, fp8=True, scaling="ntk", factor=4.0, page=128, pos=98304),
        # one request's decoded token after a short prompt: latency
        _attn("attn_token", seqs=1, new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=1000),
        # a decode batch of mixed context lengths
        _attn("attn_batch", seqs=64, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=8192),
        # verification of drafted trees over 32K contexts
        _attn("attn_trees", seqs=8, new_lo=32, new_hi=32, ctx_lo=16384, ctx_hi=32768, tree=True),
        # larger ragged trees over an e4m3 cache
        _attn("attn_trees_fp8", seqs=16, new_lo=33, new_hi=63, ctx_lo=4095, ctx_hi=16384, tree=True, fp8=True, page=128),
        # one decoded token over the 128K context
        _attn("attn_long", seqs=1, new_lo=1, new_hi=1, ctx_lo=131072, ctx_hi=131072),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "rope", "attn", "attn"])
    page = rng.choice([64, 128, 192, 256])
    if op == "extend":
        seqs = _log_int(rng, 1, 512)
        if rng.random() < 0.5:
            hi = rng.randint(1, 128)
            return dict(op=op, seqs=seqs, new_lo=rng.randint(0, hi), new_hi=hi, cache_hi=_log_int(rng, 1, 32768), page=page,
                        tree=True)
        hi = _log_int(rng, 1, max(1, 163840 // seqs))
        return dict(op=op, seqs=seqs, new_lo=rng.randint(0, hi), new_hi=hi, cache_hi=_log_int(rng, 1, 32768), page=page,
                    tree=False)
    hkv = rng.choice([1, 2, 4, 8])
    heads = dict(hq=hkv * rng.choice([1, 2, 3, 4, 5, 8]), hkv=hkv, fp8=rng.random() < 0.5, page=page)
    if op == "rope":
        scaling = rng.choice(["plain", "linear", "ntk", "yarn"])
        return dict(op=op, tokens=_log_int(rng, 1, 65536), rotary=16 * rng.randint(1, 8),
                    layout=rng.choice(["half", "interleaved"]), scaling=scaling,
                    factor=1.0 if scaling == "plain" else rng.uniform(1.5, 16.0), pos=_log_int(rng, 16, 1048576), **heads)
    seqs = _log_int(rng, 1, 64)
    tree = rng.random() < 0.6
    hi = rng.randint(1, 96) if tree else _log_int(rng, 1, 256 // min(seqs, 16))
    ctx = _log_int(rng, 1, max(2, 131072 // seqs))
    return dict(op=op, seqs=seqs, new_lo=rng.randint(1, hi), new_hi=hi, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, tree=tree,
                **heads)


# ------------------------------------------------------------------ inputs
def _spread(rng, count, lo, hi):
    """`count` lengths in lo .. hi whose sum depends on the range alone: pairs x, lo + hi - x and the middle."""
    x = rng.integers(lo, hi + 1, count // 2)
    return rng.permutation(np.concatenate([x, lo + hi - x, np.full(count % 2, (lo + hi) // 2, dtype=x.dtype)]))


def _total(case, lo="new_lo", hi="new_hi"):
    S, both = case["seqs"], case[lo] + case[hi]
    return S // 2 * both + S % 2 * (both // 2)


def _host(case, seed):
    """The integers of a case, drawn on the host: lengths, tree parents, page placement."""
    rng = np.random.default_rng([seed, 77])
    S = case["seqs"]
    new = _spread(rng, S, case["new_lo"], case["new_hi"])
    ctx = _spread(rng, S, 0, case["cache_hi"]) if case["op"] == "extend" else _spread(rng, S, case["ctx_lo"], case["ctx_hi"])
    parents = np.full(int(new.sum()), -1, dtype=np.int32)
    if case["tree"]:
        o = 0
        for n in new:
            i = np.arange(n)
            parents[o:o + n] = np.maximum(i - rng.integers(1, 7, n), 0) if n else 0
            if n:
                parents[o] = -1  # the last sampled token; the drafts descend from it
            o += n
    return rng, new.astype(np.int32), ctx.astype(np.int32), parents


def _pool(gen, pages, page, hkv, fp8, scale=None):
    x = torch.empty(pages, page, hkv, HEAD, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device="cuda")
    step = max(1, (1 << 27) // (page * hkv * HEAD))
    for p in range(0, pages, step):
        y = torch.randn(x[p:p + step].shape, generator=gen, device="cuda")
        x[p:p + step] = (y / scale[None, None, :, None]).clamp(-448, 448).to(x.dtype) if fp8 else y.to(x.dtype)
    return x


def _scales(gen, heads):
    """Per-head e4m3 scales: amax / 448 of normal data, which varies a little by head."""
    return (4.0 + torch.rand(heads, generator=gen, device="cuda")) / 448.0


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "extend":
        _prepare_extend(case, seed, st)
    elif case["op"] == "rope":
        _prepare_rope(case, seed, gen, st)
    else:
        _prepare_attn(case, seed, gen, st)
    if own:
        _bind(case, st)
    return st


def _prepare_extend(case, seed, st):
    rng, new, ctx, parents = _host(case, seed)
    S, ps = case["seqs"], case["page"]
    held = -(-ctx // ps)
    held = held + (rng.random(S) < 0.25) * (held > 0)  # some still hold a page of drafts that were rejected
    max_pages = -(-(case["cache_hi"] + case["new_hi"]) // ps) + 1
    used, extra = int(held.sum()), int(np.maximum(-(-(ctx + new) // ps) - held, 0).sum())
    pages = used + extra + 16
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((S, max_pages), -1, dtype=np.int32)
    o = 0
    for s in range(S):
        table[s, :held[s]] = order[o:o + held[s]]
        o += held[s]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    st.update(cache_lens=dev(ctx), new_lens=dev(new), held=dev(held), free=dev(order[o:]), cursor=dev(np.array([3])),
              table=dev(table), tokens=int(new.sum()) + (5 if case["tree"] else 0), pages=pages,
              words=-(-case["new_hi"] // 32) if case["tree"] else 0)
    st["parents"] = dev(np.concatenate([parents, np.full(5, -1, np.int32)])) if case["tree"] else None


def _prepare_rope(case, seed, gen, st):
    T, hq, hkv, ps = case["tokens"], case["hq"], case["hkv"], case["page"]
    # q, k and v as the fused projection leaves them: slices of one row per token
    qkv = torch.randn(T, (hq + 2 * hkv) * HEAD, generator=gen, device="cuda", dtype=torch.bfloat16)
    q, k, v = qkv.split([hq * HEAD, hkv * HEAD, hkv * HEAD], dim=1)
    pages = -(-T // ps) + 2
    rng = np.random.default_rng([seed, 78])
    first = int(rng.integers(0, max(1, case["pos"] - T + 1)))
    slots = (rng.permutation(pages)[:, None] * ps + np.arange(ps)).reshape(-1)[first % ps:][:T].astype(np.int32)
    st.update(q=q.view(T, hq, HEAD), k=k.view(T, hkv, HEAD), v=v.view(T, hkv, HEAD),
              positions=torch.arange(first, first + T, dtype=torch.int32, device="cuda"),
              slots=torch.from_numpy(slots).cuda(), q_scale=None, k_scale=None, v_scale=None)
    if case["fp8"]:
        st.update(q_scale=_scales(gen, hq), k_scale=_scales(gen, hkv), v_scale=_scales(gen, hkv))
    for n in ("k", "v"):  # the pages hold other requests' rows too
        st[n + "_pages"] = _pool(gen, pages, ps, hkv, case["fp8"], st[n + "_scale"])
    st["table"] = torch.zeros(1, pages, dtype=torch.int32, device="cuda")


def _prepare_attn(case, seed, gen, st):
    rng, new, ctx, parents = _host(case, seed)
    S, ps, hq, hkv, fp8 = case["seqs"], case["page"], case["hq"], case["hkv"], case["fp8"]
    T = int(new.sum())
    kv = ctx + new
    npg = -(-kv // ps)
    pages = int(npg.sum()) + 3
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((S, int(npg.max())), -1, dtype=np.int32)
    o = 0
    for s in range(S):
        table[s, :npg[s]] = order[o:o + npg[s]]
        o += npg[s]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    st.update(new=new.tolist(), kv=kv.tolist(), cu=cu.tolist(), q_scale=None, k_scale=None, v_scale=None, mask=None,
              table=torch.from_numpy(table).cuda(), cu_dev=torch.from_numpy(cu).cuda(),
              kv_dev=torch.from_numpy(kv.astype(np.int32)).cuda())
    q = torch.randn(T, hq, HEAD, generator=gen, device="cuda")
    if fp8:
        st.update(q_scale=_scales(gen, hq), k_scale=_scales(gen, hkv), v_scale=_scales(gen, hkv))
        st["q"] = (q / st["q_scale"][None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        st["q"] = q.to(torch.bfloat16)
    st["k_pages"] = _pool(gen, pages, ps, hkv, fp8, st["k_scale"])
    st["v_pages"] = _pool(gen, pages, ps, hkv, fp8, st["v_scale"])
    if case["tree"]:
        words = -(-case["new_hi"] // 32)
        bits = np.zeros((T, words), dtype=np.uint32)
        for s in range(S):
            for i in range(new[s]):
                j = i
                while j >= 0:
                    bits[cu[s] + i, j >> 5] |= np.uint32(1 << (j & 31))
                    j = parents[cu[s] + j]
        st["mask"] = torch.from_numpy(bits.view(np.int32)).cuda()


def _bind(case, st):
    """The descriptors and workspace that a user's program keeps beside its tensors."""
    from block_sparse_attention_stem_b200 import binding as b
    st["b"] = b
    if case["op"] == "extend":
        st["ws"] = torch.empty(256, dtype=torch.uint8, device="cuda")
        return
    st["cache"] = b.paged_kv(st["k_pages"], st["v_pages"], st["table"], case["page"])
    if case["op"] == "rope":
        st["rope"] = b.make_rope(rotary_dim=case["rotary"], layout=case["layout"], base=1e6, scaling=case["scaling"],
                                 factor=case["factor"], original_len=32768)
    else:
        st["tree"] = b.make_tree(st["q"], st["cu_dev"], st["kv_dev"], case["hkv"], mask=st["mask"],
                                 max_seq_tokens=case["new_hi"], q_scale=st["q_scale"], k_scale=st["k_scale"],
                                 v_scale=st["v_scale"])
        st["ws"] = torch.empty(b.stem_tree_ws_bytes(st["tree"]), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    if case["op"] == "extend":
        return _extend_own(st) if own else _extend_plain(st)
    if case["op"] == "rope":
        return _rope_own(st) if own else _rope_plain(st)
    return _attn_own(st) if own else _attn_plain(st)


def _extend_own(st):
    r = st["b"].stem_cache_extend(st["table"], st["case"]["page"], st["pages"], st["cache_lens"], st["new_lens"],
                                  st["held"], st["free"], st["cursor"], st["tokens"], parents=st["parents"],
                                  mask_words=st["words"], ws=st["ws"])
    out = dict(table=st["table"], held=r.held, cursor=r.cursor, cu=r.cu_seqlens, kv=r.kv_lens, slots=r.slots,
               positions=r.positions)
    if st["parents"] is not None:
        out["mask"] = r.mask
    return out


def _extend_plain(st):
    c, n, held, free, table = st["cache_lens"], st["new_lens"], st["held"], st["free"], st["table"]
    ps, T, S = st["case"]["page"], st["tokens"], c.numel()
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    cu = torch.cat([zero, n.long().cumsum(0)])
    kv = c + n
    need = (kv + ps - 1) // ps
    take = (need - held).clamp(min=0)
    base = st["cursor"].long() + torch.cat([zero, take.long().cumsum(0)])
    # table entries held .. need - 1 come from the free list, in order
    e = torch.arange(table.shape[1], device="cuda")[None, :]
    new_page = (e >= held[:, None]) & (e < need[:, None])
    idx = (base[:S, None] + e - held[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(new_page, free[idx], table))
    t = torch.arange(T, device="cuda")
    real = t < cu[S]
    s = ((t[:, None] >= cu[None, 1:]).sum(1)).clamp(max=S - 1)
    i = t - cu[s]
    p = c[s] + i
    page = table[s, (p // ps).clamp(max=table.shape[1] - 1)]
    slots = torch.where(real, page * ps + p % ps, -1).int()
    out = dict(table=table, held=torch.maximum(held, need), cursor=base[S:].int(), cu=cu.int(), kv=kv, slots=slots)
    if st["parents"] is None:
        out["positions"] = torch.where(real, p, 0).int()
        return out
    # walk every token's ancestors at once; a finished walk stays at -1
    words = st["words"]
    bits = torch.zeros(T, words, dtype=torch.int64, device="cuda")
    w = torch.arange(words, device="cuda")[None, :]
    cur = torch.where(real, i, -1)
    depth = torch.full_like(cur, -1)
    for _ in range(st["case"]["new_hi"]):
        on = cur >= 0
        bits += torch.where(on[:, None] & (w == cur[:, None] // 32), 1 << (cur[:, None].clamp(min=0) % 32), 0)
        depth += on
        cur = torch.where(on, st["parents"][(cu[s] + cur).clamp(0, T - 1)].long(), -1)
    out["positions"] = torch.where(real, c[s] + depth, 0).int()
    out["mask"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()
    return out


def _inv_freq(case):
    """Angular frequency of every rotated pair (fp64) and the amplitude."""
    r, base, f = case["rotary"], 1e6, case["factor"]
    j = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "ntk":
        base = base * f ** (r / (r - 2))
    inv = base ** (-2.0 * j / r)
    amp = 1.0
    if case["scaling"] == "linear":
        inv = inv / f
    if case["scaling"] == "yarn":
        def turn_dim(turns):  # the pair that makes `turns` turns over the trained length
            return r * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(turn_dim(32.0)), 0), min(math.ceil(turn_dim(1.0)), r - 1)
        ramp = ((j - low) / (high - low if high != low else 0.001)).clamp(0, 1)
        inv = inv / f * ramp + inv * (1 - ramp)
        amp = 0.1 * math.log(f) + 1.0
    return inv, amp


def _rope_own(st):
    q, _, _ = st["b"].stem_rope(st["rope"], st["q"], st["k"], st["v"], st["positions"], cache=st["cache"],
                                slots=st["slots"], q_scale=st["q_scale"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return dict(q=q.view(torch.float8_e4m3fn) if st["case"]["fp8"] else q, k_pages=st["k_pages"], v_pages=st["v_pages"])


def _rotate(x, cos, sin, case):
    r, h = case["rotary"], case["rotary"] // 2
    x = x.float()
    a, b = (x[..., :h], x[..., h:r]) if case["layout"] == "half" else (x[..., 0:r:2], x[..., 1:r:2])
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([u, w], -1) if case["layout"] == "half" else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _rope_plain(st):
    case = st["case"]
    inv, amp = _inv_freq(case)
    angle = st["positions"].double()[:, None] * inv
    cos, sin = (angle.cos() * amp).float()[:, None, :], (angle.sin() * amp).float()[:, None, :]

    def store(x, scale):
        if not case["fp8"]:
            return x.to(torch.bfloat16)
        return (x / scale[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)

    q = store(_rotate(st["q"], cos, sin, case), st["q_scale"])
    at = st["slots"].long()
    as_bytes = (lambda x: x.view(torch.uint8)) if case["fp8"] else (lambda x: x)
    for n, x in (("k", _rotate(st["k"], cos, sin, case)), ("v", st["v"].float())):
        as_bytes(st[n + "_pages"]).view(-1, case["hkv"], HEAD)[at] = as_bytes(store(x, st[n + "_scale"]))
    return dict(q=q, k_pages=st["k_pages"], v_pages=st["v_pages"])


def _attn_own(st):
    out, lse, _ = st["b"].stem_tree_attn(st["tree"], st["cache"], ws=st["ws"])
    return dict(out=out, lse=lse)


def _visible(st, s, n, ctx):
    """[n, n]: which of a sequence's new tokens each of them sees."""
    j = torch.arange(n, device="cuda")
    if st["mask"] is None:
        return j[None, :] <= j[:, None]
    bits = st["mask"][st["cu"][s]:st["cu"][s] + n]
    return (bits[:, j // 32] >> (j % 32)[None, :]) & 1 > 0


def _attn_plain(st):
    case = st["case"]
    hq, hkv, ps = case["hq"], case["hkv"], case["page"]
    G = hq // hkv
    T = st["cu"][-1]
    out = torch.empty(T, hq, HEAD, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(hq, T, dtype=torch.float32, device="cuda")

    def rows(name, at):
        x = st[name + "_pages"].view(-1, hkv, HEAD)
        if case["fp8"]:
            return x.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * st[name + "_scale"][None, :, None]
        return x[at].float()

    for s in range(case["seqs"]):
        n, L, o = st["new"][s], st["kv"][s], st["cu"][s]
        u = torch.arange(L, device="cuda")
        at = st["table"][s, u // ps].long() * ps + u % ps
        k, v = rows("k", at).transpose(0, 1), rows("v", at).transpose(0, 1)  # [hkv, L, d]
        q = st["q"][o:o + n].float()
        if case["fp8"]:
            q = q * st["q_scale"][None, :, None]
        q = q.view(n, hkv, G, HEAD).permute(1, 0, 2, 3).reshape(hkv, n * G, HEAD)
        x = (q @ k.transpose(1, 2)) * (HEAD ** -0.5)
        see = torch.cat([torch.ones(n, L - n, dtype=torch.bool, device="cuda"), _visible(st, s, n, L - n)], 1)
        x = torch.where(see.repeat_interleave(G, 0)[None], x, -math.inf)
        m = x.amax(2, keepdim=True)
        p = (x - m).exp()
        z = p.sum(2, keepdim=True)
        y = (p @ v) / z
        out[o:o + n] = y.view(hkv, n, G, HEAD).permute(1, 0, 2, 3).reshape(n, hq, HEAD).to(torch.bfloat16)
        lse[:, o:o + n] = (m + z.log()).view(hkv, n, G).permute(0, 2, 1).reshape(hq, n)
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    plain, st = own, None
    globals()["own"] = False
    try:
        st = prepare(case, seed)
    finally:
        globals()["own"] = plain
    return {"extend": _extend_exact, "rope": _rope_exact, "attn": _attn_exact}[case["op"]](case, st)


def _extend_exact(case, st):
    """One sequence, one page and one token at a time, on the host."""
    c, n, held, free = (st[k].tolist() for k in ("cache_lens", "new_lens", "held", "free"))
    table, cur, ps = st["table"].cpu().numpy().copy(), int(st["cursor"][0]), case["page"]
    slots, pos, cu, kv = [], [], [0], []
    mask = np.zeros((st["tokens"], max(1, st["words"])), dtype=np.uint32)
    parents = None if st["parents"] is None else st["parents"].tolist()
    for s in range(case["seqs"]):
        o = cu[-1]
        while held[s] * ps < c[s] + n[s]:
            table[s, held[s]] = free[cur]
            held[s], cur = held[s] + 1, cur + 1
        at = np.arange(c[s], c[s] + n[s])
        slots.extend((table[s, at // ps] * ps + at % ps).tolist())
        if parents is None:
            pos.extend(at.tolist())
        else:
            seen = []
            for i in range(n[s]):
                up = parents[o + i]
                seen.append((seen[up] if up >= 0 else set()) | {i})
                pos.append(c[s] + len(seen[i]) - 1)
                for j in seen[i]:
                    mask[o + i, j // 32] |= np.uint32(1 << (j % 32))
        cu.append(o + n[s])
        kv.append(c[s] + n[s])
    pad = st["tokens"] - cu[-1]
    i32 = lambda a: np.array(a, dtype=np.int32)  # noqa: E731
    out = dict(table=table, held=i32(held), cursor=i32([cur]), cu=i32(cu), kv=i32(kv), slots=i32(slots + [-1] * pad),
               positions=i32(pos + [0] * pad))
    if parents is not None:
        out["mask"] = mask.view(np.int32)
    return out


def _rope_exact(case, st):
    """Each pair as a complex number times exp(i angle)."""
    inv, amp = _inv_freq(case)
    turn = torch.polar(torch.full_like(inv, amp).expand(case["tokens"], -1), st["positions"].double()[:, None] * inv)[:, None, :]
    r = case["rotary"]

    def rotated(x, scale):
        x = x.double()
        z = x[..., :r]
        z = z.unflatten(-1, (2, r // 2)).transpose(-1, -2) if case["layout"] == "half" else z.unflatten(-1, (r // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        x[..., :r] = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
        return x if scale is None else (x / scale.double()[None, :, None]).clamp(-448, 448)

    res = dict(q=rotated(st["q"], st["q_scale"]))
    v = st["v"].double() if st["v_scale"] is None else (st["v"].double() / st["v_scale"].double()[None, :, None]).clamp(-448, 448)
    for n, x in (("k", rotated(st["k"], st["k_scale"])), ("v", v)):
        pool = st[n + "_pages"].double()
        pool.view(-1, case["hkv"], HEAD).index_copy_(0, st["slots"].long(), x)
        res[n + "_pages"] = pool
    return res


def _attn_exact(case, st):
    """One query head of one sequence at a time, each query over the keys it sees."""
    ps, G, T = case["page"], case["hq"] // case["hkv"], st["cu"][-1]
    out = torch.empty(T, case["hq"], HEAD, dtype=torch.float64, device="cuda")
    lse = torch.empty(case["hq"], T, dtype=torch.float64, device="cuda")
    for s in range(case["seqs"]):
        n, L, o = st["new"][s], st["kv"][s], st["cu"][s]
        pg = st["table"][s, :-(-L // ps)].long()
        k, v = (st[x + "_pages"][pg].flatten(0, 1)[:L].double() for x in ("k", "v"))
        hidden = torch.ones(n, L, dtype=torch.bool, device="cuda")
        hidden[:, :L - n] = False
        rowbits = None if st["mask"] is None else st["mask"][o:o + n].cpu().numpy().view(np.uint32)
        hid = np.array([[j > i if rowbits is None else not (int(rowbits[i, j >> 5]) >> (j & 31)) & 1 for j in range(n)] for i in range(n)])
        hidden[:, L - n:] = torch.from_numpy(hid).cuda()
        for h in range(case["hq"]):
            g = h // G
            f = HEAD ** -0.5 * (float(st["q_scale"][h]) * float(st["k_scale"][g]) if case["fp8"] else 1.0)
            x = (st["q"][o:o + n, h].double() @ k[:, g].T * f).masked_fill(hidden, -math.inf)
            lse[h, o:o + n] = torch.logsumexp(x, 1)
            out[o:o + n, h] = torch.exp(x - lse[h, o:o + n, None]) @ v[:, g] * (float(st["v_scale"][g]) if case["fp8"] else 1.0)
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "extend":
        S, ps = case["seqs"], case["page"]
        T = _total(case)
        words = -(-case["new_hi"] // 32) if case["tree"] else 0
        touched = T / ps + S  # pages whose numbers are read (and, if new, written to the table)
        per_token = 4 * (2 + words + (1 if case["tree"] else 0))
        return {"bytes": 4 * (6 * S + 3) + per_token * T + 8 * touched, "flops": 0}
    if case["op"] == "rope":
        T, h, hk = case["tokens"], case["hq"] + case["hkv"], case["hkv"]
        elt = 1 if case["fp8"] else 2
        return {"bytes": T * ((h + hk) * HEAD * (2 + elt) + 8), "flops": 6.0 * T * h * case["rotary"] / 2}
    S, hq, hkv, elt = case["seqs"], case["hq"], case["hkv"], 1 if case["fp8"] else 2
    T = _total(case)
    keys, rows = T + _total(case, "ctx_lo", "ctx_hi"), T * hq
    return {"bytes": keys * hkv * HEAD * 2 * elt + rows * HEAD * (elt + 2) + rows * 4 + 4 * keys / case["page"],
            "flops": 4.0 * HEAD * rows * (keys - T / 2) / S}
