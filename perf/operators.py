"""Measured cases of the rotary append and of the 8-bit paged KV cache.

Four operators: the append that rotates keys and queries on the way into the
bf16 cache; the append that also quantises to E4M3 with one scale per 64-token
tile and KV head; and decode and prefill attention over the selected blocks of
such a cache.  ``run`` makes one pass, in plain torch (``own`` false) or
through the package (``own`` true).
"""
import math

import torch

own = False

HEAD = 128
TILE = 64          # tokens that share one scale
E4M3_MAX = 448.0
MIN_EXP = -100     # least exponent of a scale


def _case(name, op, **kw):
    c = {"op": op, "decode": 0, "chunks": 0, "chunk": 0, "context": 4096, "q_heads": 64, "kv_heads": 8, "block": 64}
    if op.startswith("append"):
        c.update(rotary=128, interleaved=False, axes=1, packed=False)
    else:
        c.update(k=32)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of 8 sequences near 1M tokens: launch latency, and angles of far positions
        _case("rope_decode8_1m", "append_rope", decode=8, context=1 << 20),
        # a prefill chunk whose q, k and v are slices of one packed projection
        _case("rope_chunk4096", "append_rope", chunks=1, chunk=4096, context=135168, packed=True),
        # a mixed batch of an image model: three position axes, ragged lengths, interleaved pairs
        _case("rope_mixed_3axis", "append_rope", decode=37, chunks=2, chunk=1531, context=65536, axes=3,
              interleaved=True, block=256),
        # decode over the 8-bit cache: most tiles are partly filled, some have to be quantised anew
        _case("fp8_append_decode32", "append_fp8", decode=32, context=65536),
        # a prefill chunk into the 8-bit cache, unaligned start and length, half of the dims rotated
        _case("fp8_append_chunk1999", "append_fp8", chunks=1, chunk=1999, context=33000, rotary=64, q_heads=32,
              kv_heads=4, block=128),
        # two long chunks among decode tokens, three axes, packed projection
        _case("fp8_append_mixed", "append_fp8", decode=64, chunks=2, chunk=2048, context=131072, axes=3, packed=True),
        # the smallest call: one query, one KV head, eight blocks
        _case("fp8_decode_tiny", "decode_fp8", decode=1, context=4096, q_heads=8, kv_heads=1, k=8),
        # the decode step of a batch with long contexts
        _case("fp8_decode8_128k", "decode_fp8", decode=8, context=131072, k=32),
        # every block of a long context (dense attention as the special case), 16 heads per KV head
        _case("fp8_decode_dense64k", "decode_fp8", decode=3, context=65000, q_heads=64, kv_heads=4, k=508,
              block=128),
        # a batch of many short contexts
        _case("fp8_decode64_8k", "decode_fp8", decode=64, context=8192, q_heads=32, kv_heads=8, k=16),
        # a short prefill chunk, odd length, large blocks
        _case("fp8_prefill_333", "prefill_fp8", chunks=1, chunk=333, context=16001, q_heads=32, kv_heads=8, k=8,
              block=256),
        # the long prefill chunk after a 128K prefix
        _case("fp8_prefill_4096", "prefill_fp8", chunks=1, chunk=4096, context=135168, k=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append_rope", "append_fp8", "decode_fp8", "prefill_fp8"])
    block = rng.choice([64, 64, 128, 256, 512])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8, 16]) if kv <= 4 else rng.choice([1, 2, 4, 8])
    kw = dict(block=block, kv_heads=kv, q_heads=kv * group)
    if op.startswith("append"):
        chunks = rng.choice([0, 1, 2])
        kw.update(decode=_log_int(rng, 1, 64), chunks=chunks, chunk=_log_int(rng, 2, 2048) if chunks else 0,
                  context=_log_int(rng, 2100, 1 << 20), rotary=rng.choice([128, 128, 96, 64, 32]),
                  interleaved=rng.random() < 0.3, axes=rng.choice([1, 1, 2, 3]), packed=rng.random() < 0.5)
        return _case("", op, **kw)
    if op == "decode_fp8":
        seqs = _log_int(rng, 1, 64)
        kw.update(decode=seqs, context=_log_int(rng, 64, (1 << 20) // seqs), k=_log_int(rng, 1, 64 * TILE // block * 2))
        return _case("", op, **kw)
    chunk = _log_int(rng, 16, 1500)
    kw.update(chunks=1, chunk=chunk, context=chunk + _log_int(rng, 64, 100000), k=_log_int(rng, 1, 64 * TILE // block))
    return _case("", op, **kw)


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """(context length, new tokens) of every sequence: the chunks first; lengths are spread below the case's context."""
    new = [case["chunk"]] * case["chunks"] + [1] * case["decode"]
    spread = [0 if i < 2 else i * 2654435761 % max(1, case["context"] // 2) for i in range(len(new))]
    return [(max(case["context"] - d, n), n) for d, n in zip(spread, new)]


def _codes(shape, gen):
    """E4M3 codes of normal values that use the type's upper range."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = torch.empty(min(1 << 27, flat.numel() - i), dtype=torch.bfloat16, device="cuda")
        part.normal_(0.0, 112.0, generator=gen).clamp_(-E4M3_MAX, E4M3_MAX)
        flat[i:i + part.numel()] = part.to(torch.float8_e4m3fn)
    return out


def _scales(shape, gen, base):
    """Powers of two around 2^base, one per tile and head."""
    return torch.exp2(torch.randint(base - 1, base + 2, shape, generator=gen, device="cuda").float())


def prepare(case, seed):
    """The batch as a serving program holds it: pools, block table, lengths, queries, new rows."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    gc = torch.Generator()
    gc.manual_seed(seed)
    block, hkv, hq = case["block"], case["kv_heads"], case["q_heads"]
    seqs = _lengths(case)
    blocks = [-(-length // block) for length, _ in seqs]
    append = case["op"].startswith("append")
    # an append touches only the last blocks of each sequence: the pool holds those and some others
    kept = [min(b, -(-n // block) + 2) if append else b for b, (_, n) in zip(blocks, seqs)]
    spare = 64 * TILE // block if append else 3
    pages = sum(kept) + spare
    order = torch.randperm(pages, generator=gc)[:sum(kept)].to(torch.int32)
    table = torch.full((len(seqs), max(blocks)), -1, dtype=torch.int32)
    at = 0
    for s, (b, m) in enumerate(zip(blocks, kept)):
        table[s, b - m:b] = order[at:at + m]
        at += m
    news = [n for _, n in seqs]
    cu = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    total = int(cu[-1])
    pos = torch.cat([torch.arange(length - n, length) for length, n in seqs]).to(torch.int32)
    st = {"case": case, "table": table.cuda(), "lens": torch.tensor([length for length, _ in seqs], dtype=torch.int32).cuda(),
          "cu": cu.cuda(), "pos": pos.cuda(), "total": total,
          "kc": torch.randint(-127, 128, (pages, 64), generator=g, device="cuda", dtype=torch.int8),
          "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    shape = (pages, block, hkv, HEAD)
    tiles = (pages, block // TILE, hkv)
    if append:
        width = hq + 2 * hkv
        rows = torch.empty((total, width, HEAD), dtype=torch.bfloat16, device="cuda").normal_(0.0, 1.0, generator=g)
        # a few rows are far larger than what their tile held so far
        rows[::7] *= 4
        q, k, v = rows.split([hq, hkv, hkv], dim=1)
        if not case["packed"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        half = case["rotary"] // 2
        axes = case["axes"]
        st.update(q=q, k_new=k, v_new=v,
                  kc_new=torch.randint(-127, 128, (total, 64), generator=g, device="cuda", dtype=torch.int8),
                  inv_freq=(1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda(),
                  pair_axis=None, axis_pos=None, q_out=torch.empty((total, hq, HEAD), dtype=torch.bfloat16, device="cuda"))
        if axes > 1:
            # the first quarter of the pairs turns with time, the rest with height and width
            bounds = [half // 4 if axes == 3 else half // 2, half - (half - half // 4) // 2]
            idx = torch.arange(half)
            st["pair_axis"] = ((idx >= bounds[0]).int() + ((idx >= bounds[1]).int() if axes == 3 else 0)).int().cuda()
            grid = torch.randint(0, 128, (axes - 1, total), generator=g, device="cuda", dtype=torch.int32)
            st["axis_pos"] = torch.cat([st["pos"][None], st["pos"][None] // 4 + grid]).contiguous()
        if case["op"] == "append_rope":
            for n in ("k_pool", "v_pool"):
                st[n] = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, 1.0, generator=g)
        else:
            for n in ("k", "v"):
                st[n + "_pool"] = _codes(shape, g)
                st[n + "_scale"] = _scales(tiles, g, -7)
    else:
        st["k_pool"], st["v_pool"] = _codes(shape, g), _codes(shape, g)
        st["k_scale"], st["v_scale"] = _scales(tiles, g, -7), _scales(tiles, g, -7)
        st["q"] = torch.empty((total, hq, HEAD), dtype=torch.bfloat16, device="cuda").normal_(0.0, 2.0, generator=g)
        seq = torch.repeat_interleave(torch.arange(len(seqs)), torch.tensor(news)).cuda()
        own_block = (st["pos"] // block).long()
        k = case["k"]
        # distinct blocks in ascending order, the query's own among them, -1 behind the last
        score = torch.rand((total, table.shape[1]), generator=g, device="cuda")
        col = torch.arange(table.shape[1], device="cuda")
        score[col[None] > own_block[:, None]] = -1.0
        score.scatter_(1, own_block[:, None], 2.0)
        best, ids = score.topk(min(k, score.shape[1]), dim=1)
        ids = torch.where(best >= 0, ids, 1 << 30).sort(dim=1).values
        sel = torch.full((total, k), -1, dtype=torch.int32, device="cuda")
        sel[:, :ids.shape[1]] = torch.where(ids == 1 << 30, -1, ids).int()
        st.update(sel=sel, cnt=(sel >= 0).sum(1).int(), seq=seq, out=torch.empty_like(st["q"]),
                  lse=torch.empty((total, hq), device="cuda"))
        # zero before its first use, as the call wants it; kept from step to step
        st["workspace"] = torch.zeros(total * hkv * 4 + 256 + 2 * 256 * (hq // hkv) * 132 * 4 + 256, dtype=torch.uint8,
                                      device="cuda")
    return st


# ---------------------------------------------------------------- plain forms

def _seq_of(st, dtype=torch.int64):
    return torch.searchsorted(st["cu"][1:].to(dtype), torch.arange(st["total"], device="cuda"), right=True)


def _angles(st):
    """[tokens][pairs] angles in 64 bits."""
    pos = st["pos"][None] if st["axis_pos"] is None else st["axis_pos"]
    half = st["case"]["rotary"] // 2
    axis = torch.zeros(half, dtype=torch.int64, device="cuda") if st["pair_axis"] is None else st["pair_axis"].long()
    return pos.double()[axis].t() * st["inv_freq"].double()


def _rotate(x, cos, sin, case):
    rd = case["rotary"]
    cos, sin = cos[:, None], sin[:, None]
    turned, rest = x[..., :rd], x[..., rd:]
    if case["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = turned[..., :rd // 2], turned[..., rd // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _coarse_keys(st, seq, page):
    """The last new row of each touched block."""
    ends = torch.ones(st["total"], dtype=torch.bool, device="cuda")
    ends[:-1] = (seq[1:] != seq[:-1]) | (page[1:] != page[:-1])
    # rows that are not the last of their block write what the last one writes
    last = torch.where(ends, torch.arange(st["total"], device="cuda"), st["total"])
    last = last.flip(0).cummin(0).values.flip(0)
    st["kc"][page] = st["kc_new"][last]


def _append_plain(st):
    case, block = st["case"], st["case"]["block"]
    seq = _seq_of(st)
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    pos = st["lens"].long()[seq] - n[seq] + torch.arange(st["total"], device="cuda") - st["cu"].long()[seq]
    page = st["table"][seq, pos // block].long()
    slot = pos % block
    ang = _angles(st)
    cos, sin = ang.cos().float(), ang.sin().float()
    q = _rotate(st["q"].float(), cos, sin, case).bfloat16()
    k = _rotate(st["k_new"].float(), cos, sin, case)
    v = st["v_new"].float()
    _coarse_keys(st, seq, page)
    if case["op"] == "append_rope":
        st["k_pool"][page, slot] = k.bfloat16()
        st["v_pool"][page, slot] = v.bfloat16()
        return {"q": q, "k": st["k_pool"], "v": st["v_pool"], "kc": st["kc"]}
    # every touched tile, some of them twice: this many places hold any batch of as many tokens and sequences
    first = st["lens"].long() - n
    base = st["cu"][:-1].long() // TILE + 2 * torch.arange(len(n), device="cuda")
    u = torch.arange(st["total"] // TILE + 2 * len(n), device="cuda")
    s = torch.searchsorted(base, u, right=True) - 1
    start = torch.minimum((first[s] // TILE + u - base[s]) * TILE, (st["lens"].long()[s] - 1) // TILE * TILE)
    tpage, tsub = st["table"][s, start // block].long(), start % block // TILE
    kept = (first[s] - start).clamp(0, TILE)          # tokens the tile held before
    where = start // TILE - first[s] // TILE + base[s]  # a tile's place: the first that names it
    mine = pos // TILE - first[seq] // TILE + base[seq]
    slots = torch.arange(TILE, device="cuda")
    for name, x in (("k", k), ("v", v)):
        pool, scale = st[name + "_pool"], st[name + "_scale"]
        mag = torch.zeros((len(u), case["kv_heads"]), device="cuda")
        mag.index_reduce_(0, mine, x.abs().amax(-1), "amax")
        mag = mag[where]
        m, e = torch.frexp(mag)                        # mag = m 2^e with m in [1/2, 1); 448 = 0.875 * 2^9
        need = torch.where(mag > 0, (e - 9 + (m > 0.875)).clamp(min=MIN_EXP), MIN_EXP).float().exp2()
        old = scale[tpage, tsub]
        new = torch.where((kept > 0)[:, None], torch.maximum(old, need), need)
        tiled = pool.view(torch.uint8).view(pool.shape[0], block // TILE, TILE, *pool.shape[2:])
        held = tiled[tpage, tsub].view(torch.float8_e4m3fn)
        again = (held.float() * (old / new)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        keep = (slots[None] < kept[:, None])[:, :, None, None]
        tiled[tpage, tsub] = torch.where(keep, again.view(torch.uint8), held.view(torch.uint8))
        scale[tpage, tsub] = new
        code = (x / new[mine][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        pool.view(torch.uint8)[page, slot] = code.view(torch.uint8)
    return _fp8_outputs(st, q)


def _fp8_outputs(st, q):
    return {"q": q, "k": st["k_pool"], "v": st["v_pool"], "ks": st["k_scale"], "vs": st["v_scale"], "kc": st["kc"]}


def _attention_part(st, lo, hi):
    case, block = st["case"], st["case"]["block"]
    hkv, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    sel = st["sel"][lo:hi].long()
    t, k = sel.shape
    page = st["table"][st["seq"][lo:hi, None], sel.clamp(min=0)].long()

    def rows(pool, scale):
        x = pool.view(torch.uint8)[page].view(torch.float8_e4m3fn).float()
        x = x.view(t, k, block // TILE, TILE, hkv, HEAD) * scale[page][:, :, :, None, :, None]
        return x.view(t, k * block, hkv, HEAD).transpose(1, 2)

    q = st["q"][lo:hi].float().view(t, hkv, group, HEAD)
    score = q @ rows(st["k_pool"], st["k_scale"]).transpose(2, 3) / math.sqrt(HEAD)
    tok = (sel * block)[:, :, None] + torch.arange(block, device="cuda")
    seen = ((sel >= 0)[:, :, None] & (tok <= st["pos"][lo:hi].long()[:, None, None])).view(t, 1, 1, k * block)
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    norm = p.sum(-1, keepdim=True)
    out = (p @ rows(st["v_pool"], st["v_scale"])) / norm
    return out.reshape(t, case["q_heads"], HEAD).bfloat16(), (top + norm.log()).view(t, case["q_heads"])


def _attention_plain(st):
    # the gathered rows of all queries together do not fit: a part of the queries at a time
    case = st["case"]
    step = max(1, (1 << 28) // (case["k"] * case["block"] * case["kv_heads"] * HEAD))
    parts = [_attention_part(st, lo, min(lo + step, st["total"])) for lo in range(0, st["total"], step)]
    return {"out": torch.cat([o for o, _ in parts]), "lse": torch.cat([x for _, x in parts])}


# ---------------------------------------------------------------- the package's calls

def _run_own(st):
    import dynamic_block_sparse_dsa_b200 as dsa
    case = st["case"]
    seqs = dsa.SeqBatch(st["table"], st["lens"])
    queries = dsa.QueryBatch(st["cu"], st["pos"])
    if case["op"] == "append_rope":
        cache = dsa.PagedKVCache(st["k_pool"], st["v_pool"], st["kc"])
    else:
        cache = dsa.PagedKVCacheFP8(st["k_pool"], st["v_pool"], st["kc"], st["k_scale"], st["v_scale"])
    if case["op"].startswith("append"):
        rope = dsa.Rotary(st["inv_freq"], interleaved=case["interleaved"], num_axes=case["axes"],
                          pair_axis=st["pair_axis"])
        call = dsa.kv_append_rope if case["op"] == "append_rope" else dsa.kv_append_fp8
        q = call(cache, seqs, st["cu"], st["k_new"], st["v_new"], st["kc_new"], rope, pos_new=st["axis_pos"],
                 queries=queries, q=st["q"], pos_q=st["axis_pos"], q_out=st["q_out"], dev_err=st["err"])
        if case["op"] == "append_rope":
            return {"q": q, "k": st["k_pool"], "v": st["v_pool"], "kc": st["kc"]}
        return _fp8_outputs(st, q)
    if case["op"] == "decode_fp8":
        out, lse = dsa.sparse_attn_decode_fp8(cache, seqs, queries, st["q"], st["sel"], st["cnt"], out=st["out"],
                                              lse=st["lse"], workspace=st["workspace"], dev_err=st["err"])
    else:
        out, lse = dsa.sparse_attn_prefill_fp8(cache, seqs, queries, st["q"], st["sel"], st["cnt"], out=st["out"],
                                               lse=st["lse"], dev_err=st["err"])
    return {"out": out, "lse": lse}


def run(st):
    if own:
        return _run_own(st)
    if st["case"]["op"].startswith("append"):
        return _append_plain(st)
    return _attention_plain(st)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_append(case, st):
    """Token by token positions on the host, tiles from their definition."""
    block, rd = case["block"], case["rotary"]
    cu, lens, table = st["cu"].tolist(), st["lens"].tolist(), st["table"].cpu()
    where, page, slot, tiles = [], [], [], {}
    kc = st["kc"].clone()
    for s in range(len(lens)):
        n = cu[s + 1] - cu[s]
        for i in range(n):
            p = lens[s] - n + i
            pg = int(table[s, p // block])
            where.append(p)
            page.append(pg)
            slot.append(p % block)
            tiles.setdefault((pg, p % block // TILE), []).append(cu[s] + i)
    page_t, slot_t = torch.tensor(page).cuda(), torch.tensor(slot).cuda()
    last = {}
    for i, pg in enumerate(page):
        last[pg] = i
    kc[torch.tensor(list(last.keys())).cuda()] = st["kc_new"][torch.tensor(list(last.values())).cuda()]
    pos = torch.tensor(where, dtype=torch.float64)[None] if st["axis_pos"] is None else st["axis_pos"].double().cpu()
    axis = [0] * (rd // 2) if st["pair_axis"] is None else st["pair_axis"].tolist()
    ang = torch.stack([pos[axis[i]] * float(st["inv_freq"][i]) for i in range(rd // 2)], dim=1).cuda()

    def turn(x):
        y = x.double().clone()
        i = torch.arange(rd // 2, device="cuda")
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rd // 2)
        z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones_like(ang), ang)[:, None]
        y[..., a], y[..., b] = z.real, z.imag
        return y

    q, k, v = turn(st["q"]), turn(st["k_new"]), st["v_new"].double()
    if case["op"] == "append_rope":
        kp, vp = st["k_pool"].double(), st["v_pool"].double()
        kp[page_t, slot_t], vp[page_t, slot_t] = k, v
        return {"q": q, "k": kp, "v": vp, "kc": kc}
    got = {"q": q, "kc": kc}
    for name, x in (("k", k), ("v", v)):
        pool, scale = st[name + "_pool"].double(), st[name + "_scale"].double()
        for (pg, sub), ids in tiles.items():
            begin = slot[ids[0]] - sub * TILE
            mag = x[ids].abs().amax(dim=(0, 2))
            need = torch.exp2(torch.ceil(torch.log2((mag / E4M3_MAX).clamp(min=2.0 ** MIN_EXP))))
            was = scale[pg, sub].clone()
            now = need if begin == 0 else torch.maximum(was, need)
            rows = pool[pg, sub * TILE:(sub + 1) * TILE]
            rows[:begin] *= (was / now)[:, None]
            rows[begin:begin + len(ids)] = x[ids] / now[:, None]
            scale[pg, sub] = now
        got[name], got[name + "s"] = pool, scale
    return got


def _exact_attention(case, st):
    block, hq, hkv = case["block"], case["q_heads"], case["kv_heads"]
    group = hq // hkv
    sel, cnt = st["sel"].cpu(), st["cnt"].tolist()
    pos, seq, table = st["pos"].tolist(), st["seq"].tolist(), st["table"]
    out = torch.zeros((st["total"], hq, HEAD), dtype=torch.float64, device="cuda")
    lse = torch.full((st["total"], hq), -math.inf, dtype=torch.float64, device="cuda")
    offs = torch.arange(block, device="cuda")
    for t in range(st["total"]):
        ids = sel[t, :cnt[t]].long().cuda()
        pages = table[seq[t]][ids].long()
        see = (ids[:, None] * block + offs).flatten() <= pos[t]
        ks = st["k_scale"][pages].double().repeat_interleave(TILE, dim=1)
        vs = st["v_scale"][pages].double().repeat_interleave(TILE, dim=1)
        k = (st["k_pool"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double() * ks[..., None]).flatten(0, 1)
        v = (st["v_pool"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double() * vs[..., None]).flatten(0, 1)
        k, v = k[see].transpose(0, 1), v[see].transpose(0, 1)
        s = torch.bmm(st["q"][t].double().view(hkv, group, HEAD), k.transpose(1, 2)) / math.sqrt(HEAD)
        lse[t] = torch.logsumexp(s, dim=2).flatten()
        out[t] = torch.bmm(torch.softmax(s, dim=2), v).reshape(hq, HEAD)
    return {"out": out, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(case, st) if case["op"].startswith("append") else _exact_attention(case, st)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    seqs, hq, hkv, block = _lengths(case), case["q_heads"], case["kv_heads"], case["block"]
    total = sum(n for _, n in seqs)
    if case["op"].startswith("append"):
        out_row = 2 * hkv * HEAD * (2 if case["op"] == "append_rope" else 1)
        tiles = sum((length - 1) // TILE - (length - n) // TILE + 1 for length, n in seqs)
        scales = 0 if case["op"] == "append_rope" else 2 * tiles * hkv * 4
        nbytes = total * (2 * hq * HEAD * 2 + 2 * hkv * HEAD * 2 + out_row + 64 + 4 * case["axes"]) + scales
        return {"bytes": nbytes, "flops": total * (hq + hkv) * case["rotary"] * 3}
    seen = pairs = 0
    for length, n in seqs:
        each = [min(p + 1, case["k"] * block) for p in range(length - n, length)]
        pairs += sum(each)
        seen += min(length, sum(each))
    nbytes = seen * hkv * (2 * HEAD + 8 / TILE) + total * hq * (4 * HEAD + 4) + total * case["k"] * 4
    return {"bytes": nbytes, "flops": 4 * pairs * hq * HEAD}
