"""Rotary append and the 8-bit cache on the GPU, against plain float64 versions
of the same definitions (rope_fp8_reference.py, which also derives the
tolerances used here)."""
import math

import pytest
import torch

import dynamic_block_sparse_dsa_b200 as dsa
from dynamic_block_sparse_dsa_b200 import _lib

import rope_fp8_reference as ref

pytestmark = pytest.mark.gpu

BF16_HALF, E4M3_HALF = 2.0 ** -8, 2.0 ** -4


class Batch:
    """Ragged sequences over a shuffled pool: lens after the append, n_new new tokens each."""

    def __init__(self, lens, n_new, hkv, hq, block=64, seed=0, packed=False, spare=3, v_big=1.0):
        g = torch.Generator().manual_seed(seed)
        self.block, self.hkv, self.hq = block, hkv, hq
        nb = [-(-L // block) for L in lens]
        self.pages = sum(nb) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = torch.full((len(lens), max(max(nb), 1)), -1, dtype=torch.int32)
        at = 0
        for s, b in enumerate(nb):
            self.table[s, :b] = torch.tensor(order[at:at + b], dtype=torch.int32)
            at += b
        self.lens = list(lens)
        self.cu = [0]
        for n in n_new:
            self.cu.append(self.cu[-1] + n)
        T = self.T = self.cu[-1]
        width = hq + 2 * hkv
        rows = torch.randn(T, width, 128, generator=g)
        rows *= torch.exp2(torch.randint(-3, 4, (T, 1, 1), generator=g).float())   # scales that have to grow
        rows = rows.bfloat16()
        q, k, v = rows.split([hq, hkv, hkv], dim=1)
        dev = rows.cuda()
        dq, dk, dv = dev.split([hq, hkv, hkv], dim=1)
        if not packed:
            dq, dk, dv = dq.contiguous(), dk.contiguous(), dv.contiguous()
        self.q, self.k, self.v, self.dq, self.dk, self.dv = q, k, v, dq, dk, dv
        self.kc = torch.randint(-127, 128, (T, 64), generator=g, dtype=torch.int8)
        self.kc_pool = torch.randint(-127, 128, (self.pages, 64), generator=g, dtype=torch.int8)
        self.spots = ref.places(self.table, self.lens, self.cu, block)
        self.pos = torch.tensor([p for _, p, _, _ in self.spots], dtype=torch.int32)
        self.seq = [s for s, _, _, _ in self.spots]
        self.gen = g
        self.seqs = dsa.SeqBatch(self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda())
        self.queries = dsa.QueryBatch(torch.tensor(self.cu, dtype=torch.int32).cuda(), self.pos.cuda())
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def shape(self):
        return (self.pages, self.block, self.hkv, 128)

    def cache16(self):
        k, v = (torch.randn(self.shape(), generator=self.gen).bfloat16() for _ in range(2))
        return (k, v), dsa.PagedKVCache(k.cuda(), v.cuda(), self.kc_pool.cuda())

    def cache8(self, nan_slots=False, spread=2):
        """(host codes and scales, device cache): random codes (no NaN unless nan_slots fills
        the slots behind each sequence with NaN codes), power-of-two scales."""
        host = []
        for _ in range(2):
            c = ref.encode_e4m3(torch.randn(self.shape(), generator=self.gen).double() * 100)
            if nan_slots:
                for s, L in enumerate(self.lens):
                    if L % self.block:
                        c[int(self.table[s][L // self.block]), L % self.block:] = 0x7F
                used = self.table[self.table >= 0].tolist()
                for pg in set(range(self.pages)) - set(used):
                    c[pg] = 0xFF
            s = torch.exp2(torch.randint(-7 - spread, -6 + spread, (self.pages, self.block // 64, self.hkv),
                                         generator=self.gen).float())
            host.append((c, s))
        (k, ks), (v, vs) = host
        return host, dsa.PagedKVCacheFP8(k.cuda(), v.cuda(), self.kc_pool.cuda(), ks.cuda(), vs.cuda())

    def kc_after(self):
        kc = self.kc_pool.clone()
        for i, (_, _, pg, _) in enumerate(self.spots):
            kc[pg] = self.kc[i]
        return kc


def freqs(half, base=1e4):
    return (base ** (-torch.arange(half, dtype=torch.float64) / half)).float()


def rotary(rd=128, interleaved=False, axes=1, scale=1.0):
    inv = freqs(rd // 2)
    axis = None if axes == 1 else (torch.arange(rd // 2, dtype=torch.int32) * axes // (rd // 2)).int()
    return inv, axis, dsa.Rotary(inv.cuda(), interleaved, axes, None if axis is None else axis.cuda(), scale)


def check_rows(got, want, slack, step, floor=0.0):
    d = (got.double() - want).abs()
    tol = want.abs() * step + slack * (1 + step) + floor
    bad = d > tol
    assert not bool(bad.any()), (float((d - tol).max()), int(bad.sum()))


APPENDS = {
    # name: lens, n_new, hkv, hq, block, rotation, packed
    "decode": dict(lens=(1, 65, 4096, 640), n_new=(1, 1, 1, 1), hkv=2, hq=16),
    "none_and_one": dict(lens=(70, 3, 128), n_new=(0, 3, 0), hkv=1, hq=1),
    "ragged_chunks": dict(lens=(300, 64, 131, 1000), n_new=(137, 64, 3, 0), hkv=3, hq=15, packed=True),
    "pages_of_256": dict(lens=(700, 257, 512), n_new=(600, 2, 1), hkv=2, hq=8, block=256),
    "interleaved_half": dict(lens=(200, 90), n_new=(150, 1), hkv=2, hq=6, rot=dict(rd=64, interleaved=True),
                             packed=True),
    "three_axes": dict(lens=(260,), n_new=(130,), hkv=4, hq=8, block=128, rot=dict(rd=96, axes=3)),
    "scaled_16dims": dict(lens=(80, 80), n_new=(40, 7), hkv=8, hq=72, rot=dict(rd=16, scale=0.75)),
    "many_seqs": dict(lens=tuple(range(1, 301)), n_new=tuple(i % 3 for i in range(300)), hkv=1, hq=2),
    "many_heads": dict(lens=(130,), n_new=(1,), hkv=70, hq=70),
}


def make(name, seed=3):
    kw = dict(APPENDS[name])
    rot = kw.pop("rot", {})
    b = Batch(seed=seed, **kw)
    inv, axis, rope = rotary(**rot)
    axes = rot.get("axes", 1)
    pos = None
    if axes > 1:
        pos = torch.stack([b.pos] + [torch.randint(0, 90, (b.T,), generator=b.gen, dtype=torch.int32)
                                     for _ in range(axes - 1)])
    hpos = b.pos[None] if pos is None else pos
    turn = lambda x: ref.rotate(x.double(), hpos, inv, rot.get("interleaved", False), axis, rot.get("scale", 1.0))  # noqa: E731
    return b, rope, None if pos is None else pos.cuda(), turn


@pytest.mark.parametrize("name", sorted(APPENDS))
def test_append_rope(name, cuda_device):
    b, rope, pos, turn = make(name)
    (k0, v0), cache = b.cache16()
    q = dsa.kv_append_rope(cache, b.seqs, b.queries.cu_q, b.dk, b.dv, b.kc.cuda(), rope, pos_new=pos, queries=b.queries,
                           q=b.dq, pos_q=pos, dev_err=b.err)
    assert int(b.err) == 0
    want, slack = turn(b.q)
    check_rows(q.cpu(), want, slack, BF16_HALF)
    rd = 2 * rope.inv_freq.numel()
    assert torch.equal(q.cpu()[:, :, rd:], b.q[:, :, rd:])
    kw, ks = turn(b.k)
    k, v = cache.k_pool.cpu(), cache.v_pool.cpu()
    for i, (_, _, pg, slot) in enumerate(b.spots):
        check_rows(k[pg, slot], kw[i], ks[i], BF16_HALF)
        assert torch.equal(k[pg, slot, :, rd:], b.k[i, :, rd:])
        assert torch.equal(v[pg, slot], b.v[i])
        k[pg, slot], v[pg, slot] = k0[pg, slot], v0[pg, slot]
    assert torch.equal(k, k0) and torch.equal(v, v0)     # every other row as it was
    assert torch.equal(cache.kc_pool.cpu(), b.kc_after())


def check_fp8_append(b, host, cache, kw, kslack):
    """Pools, scales and coarse keys after an append of (rotated) rows kw with slack kslack."""
    for (c0, s0), pool, scale, x, slack in ((host[0], cache.k_pool, cache.k_scale, kw, kslack),
                                            (host[1], cache.v_pool, cache.v_scale, b.v.double(), None)):
        c, s = pool.cpu(), scale.cpu()
        for (pg, sub), (first, ids, was, now) in ref.append_tiles(c0, s0, x, b.spots, b.cu).items():
            assert torch.equal(s[pg, sub].double(), now), (pg, sub)
            rows = slice(sub * 64, sub * 64 + first)
            again = ref.encode_e4m3(ref.decode_e4m3(c0[pg, rows]) * (was / now)[None, :, None])
            held = torch.where((was == now)[None, :, None], c0[pg, rows], again)
            assert torch.equal(ref.decode_e4m3(c[pg, rows]), ref.decode_e4m3(held))
            for n, i in enumerate(ids):
                slot = sub * 64 + first + n
                if slack is None:      # no rotation: the code is the conversion of the value itself
                    assert torch.equal(ref.decode_e4m3(c[pg, slot]), ref.decode_e4m3(ref.encode_e4m3(x[i] / now[:, None])))
                else:
                    check_rows(ref.decode_e4m3(c[pg, slot]) * now[:, None], x[i], slack[i], E4M3_HALF,
                               floor=now[:, None] * 2.0 ** -10)
                c[pg, slot] = c0[pg, slot]
            c[pg, rows] = c0[pg, rows]
            s[pg, sub] = s0[pg, sub]
        assert torch.equal(c, c0) and torch.equal(s, s0)
    assert torch.equal(cache.kc_pool.cpu(), b.kc_after())


@pytest.mark.parametrize("turned", [True, False], ids=["rotated", "as_is"])
@pytest.mark.parametrize("name", sorted(APPENDS))
def test_append_fp8(name, turned, cuda_device):
    b, rope, pos, turn = make(name, seed=4)
    host, cache = b.cache8()
    if turned:
        q = dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q, b.dk, b.dv, b.kc.cuda(), rope, pos_new=pos,
                              queries=b.queries, q=b.dq, pos_q=pos, dev_err=b.err)
        want, slack = turn(b.q)
        check_rows(q.cpu(), want, slack, BF16_HALF)
        kw, ks = turn(b.k)
    else:
        assert dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q, b.dk, b.dv, b.kc.cuda(), dev_err=b.err) is None
        kw, ks = b.k.double(), torch.zeros(b.k.shape, dtype=torch.float64)
    assert int(b.err) == 0
    check_fp8_append(b, host, cache, kw, ks)


def test_append_fp8_token_by_token_grows_the_scale(cuda_device):
    """64 tokens one at a time, each twice as large as the last for a while: the scale
    follows the largest so far, and earlier rows keep their value to the codes' rounding."""
    b = Batch((64,), (64,), 1, 1, seed=9)
    mag = torch.exp2((torch.arange(64) % 20).float() - 10)
    x = (torch.rand(64, 1, 128, generator=b.gen) * 0.9 + 0.1) * mag[:, None, None]
    x = x.bfloat16()
    _, cache = b.cache8()
    cache.k_scale.fill_(float("nan"))          # never written: the first token of a tile sets it
    cache.v_scale.fill_(float("inf"))
    table, cu = b.seqs.block_table, torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for i in range(64):
        s = dsa.SeqBatch(table, torch.tensor([i + 1], dtype=torch.int32, device="cuda"))
        dsa.kv_append_fp8(cache, s, cu, x[i:i + 1].cuda(), x[i:i + 1].cuda(), dev_err=b.err)
    assert int(b.err) == 0
    pg = int(b.table[0, 0])
    for pool, scale in ((cache.k_pool, cache.k_scale), (cache.v_pool, cache.v_scale)):
        now = float(scale[pg, 0, 0])
        assert now == ref.need_of(float(x.abs().max()))
        got = ref.decode_e4m3(pool[pg].cpu()) * now
        # one rounding to 4 bits; a code that became subnormal on the way may round again, each
        # time by at most half the subnormal step of that scale: their sum is below a whole step
        check_rows(got, x.double(), torch.zeros_like(x).double(), E4M3_HALF, floor=now * 2.0 ** -9)


def test_append_far_positions_and_in_place_queries(cuda_device):
    """Positions to the end of int32 and below zero; q rotated in place; no new tokens."""
    b = Batch((5,), (5,), 1, 4, seed=11)
    pos = torch.tensor([0, -1, 1048575, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64)
    inv, _, rope = rotary()
    q = b.dq.clone()
    p32 = pos.to(torch.int32).cuda()
    (k0, v0), cache = b.cache16()
    got = dsa.kv_append_rope(cache, b.seqs, None, None, None, None, rope, queries=b.queries, q=q, pos_q=p32[None],
                             q_out=q, dev_err=b.err)
    assert got is q and int(b.err) == 0
    want, slack = ref.rotate(b.q.double(), pos[None], inv)
    # the turn fraction of f = inv_freq / 2 pi is off by 2^-53 f a position: 2^-22 of a turn at 2^31, 1.5e-6 rad
    check_rows(q.cpu(), want, slack + b.q.double().abs().amax(2, keepdim=True) * 2.0 ** -18, BF16_HALF)
    assert torch.equal(cache.k_pool.cpu(), k0) and torch.equal(cache.v_pool.cpu(), v0)


def test_append_fp8_values_at_the_edges(cuda_device):
    """Zeros, the exact border 448 * 2^e and the next value up, infinities, NaN, tiny values."""
    b = Batch((8,), (8,), 1, 1, seed=12)
    x = torch.zeros(8, 1, 128)
    x[1] = 448.0 * 2.0 ** -3
    x[2, 0, 5] = 2.0 ** -126
    b_v = x.bfloat16()
    _, cache = b.cache8()
    cu = b.queries.cu_q
    dsa.kv_append_fp8(cache, b.seqs, cu, b_v.cuda(), torch.zeros_like(b_v).cuda(), dev_err=b.err)
    pg = int(b.table[0, 0])
    assert int(b.err) == 0
    assert float(cache.k_scale[pg, 0, 0]) == 2.0 ** -3 and float(cache.v_scale[pg, 0, 0]) == 2.0 ** -100
    assert torch.equal(ref.decode_e4m3(cache.k_pool[pg, 1].cpu()), torch.full((1, 128), 448.0, dtype=torch.float64))
    assert not bool(cache.v_pool[pg, :8].any())
    y = b_v.clone()
    y[1, 0, 0] = 450.0 * 2.0 ** -3           # bf16 keeps 8 bits: 450 is representable, one step above 448
    y[3, 0, 1], y[3, 0, 2], y[3, 0, 3] = math.inf, -math.inf, math.nan
    dsa.kv_append_fp8(cache, b.seqs, cu, y.cuda(), y.cuda(), dev_err=b.err)
    assert int(b.err) == _lib.DEV_ERR_VALUE
    for pool, scale in ((cache.k_pool, cache.k_scale), (cache.v_pool, cache.v_scale)):
        assert float(scale[pg, 0, 0]) == 2.0 ** -2
        row = ref.decode_e4m3(pool[pg, 3, 0].cpu())
        assert row[1] == 448 and row[2] == -448 and bool(row[3].isnan()) and not bool(row[4:].any())


def test_append_bad_descriptions_are_reported_and_skipped(cuda_device):
    """A page outside the pool, more new tokens than the sequence has, a table too short, an
    axis out of range: the bit is set, nothing else is written, the other sequences get theirs."""
    for kind, bit in (("page", _lib.DEV_ERR_PAGE), ("len", _lib.DEV_ERR_POS), ("table", _lib.DEV_ERR_POS),
                      ("total", _lib.DEV_ERR_POS)):
        for fp8 in (False, True):
            b = Batch((70, 100, 66), (3, 4, 66), 2, 4, seed=13)
            inv, _, rope = rotary()
            host, cache = b.cache8() if fp8 else b.cache16()
            before = [t.clone() for t in (cache.k_pool, cache.v_pool)]
            table, lens, cu = b.table.clone(), list(b.lens), torch.tensor(b.cu, dtype=torch.int32)
            if kind == "page":
                table[1, 1] = b.pages
            elif kind == "len":
                lens[1] = 3
            elif kind == "table":
                lens[1] = 64 * table.shape[1] + 4
            else:
                cu[3] -= 1                       # the last new token belongs to no sequence
                lens[2] -= 1
            seqs = dsa.SeqBatch(table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
            call = dsa.kv_append_fp8 if fp8 else dsa.kv_append_rope
            call(cache, seqs, cu.cuda(), b.dk, b.dv, b.kc.cuda(), rope, dev_err=b.err)
            assert int(b.err) == bit, (kind, fp8, int(b.err))
            for i, (s, _, pg, slot) in enumerate(b.spots):
                skipped = i == b.T - 1 if kind == "total" else s == 1
                assert torch.equal(cache.v_pool[pg, slot], before[1][pg, slot]) == skipped, (kind, fp8, i)
    b = Batch((70,), (3,), 2, 4, seed=14)
    inv, _, rope = rotary(axes=2)
    rope.pair_axis[3] = 2
    _, cache = b.cache16()
    pos = torch.stack([b.pos, b.pos]).cuda()
    q = dsa.kv_append_rope(cache, b.seqs, b.queries.cu_q, b.dk, b.dv, None, rope, pos_new=pos, queries=b.queries, q=b.dq,
                           pos_q=pos, dev_err=b.err)
    assert int(b.err) == _lib.DEV_ERR_POS
    want, slack = ref.rotate(b.q.double(), b.pos[None], inv)
    check_rows(q.cpu(), want, slack, BF16_HALF)


# ----------------------------------------------------------------------------- attention

ATTN = {
    "one_token": dict(lens=(1,), n_new=(1,), hkv=1, hq=1, k=1),
    "one_block": dict(lens=(37, 64), n_new=(1, 2), hkv=2, hq=2, k=4),
    "group8": dict(lens=(700, 130, 1500), n_new=(1, 1, 1), hkv=2, hq=16, k=6),
    "group16": dict(lens=(900,), n_new=(3,), hkv=2, hq=32, k=9),
    "group5": dict(lens=(333, 200), n_new=(5, 1), hkv=3, hq=15, k=3),
    "group11": dict(lens=(400,), n_new=(2,), hkv=1, hq=11, k=7),
    "pages_of_128": dict(lens=(1000, 129), n_new=(2, 1), hkv=2, hq=8, k=3, block=128),
    "pages_of_512": dict(lens=(1500, 700), n_new=(1, 3), hkv=1, hq=8, k=2, block=512),
    "chunk": dict(lens=(500,), n_new=(70,), hkv=2, hq=8, k=3),
    # 48 (query, KV head) pairs: a cluster of two per pair
    "clusters": dict(lens=tuple(range(70, 70 + 24 * 41, 41)), n_new=(1,) * 24, hkv=2, hq=4, k=5),
    "whole_context": dict(lens=(3000,), n_new=(1,), hkv=2, hq=8, k=47),
}


def selection(b, k, own=True):
    sel = torch.full((b.T, k), -1, dtype=torch.int32)
    cnt = torch.zeros(b.T, dtype=torch.int32)
    for t in range(b.T):
        last = int(b.pos[t]) // b.block
        ids = torch.randperm(last, generator=b.gen)[:k - 1].tolist() + [last]
        ids = sorted(ids)[:k]
        sel[t, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
        cnt[t] = len(ids)
    return sel, cnt


def attend(b, cache, q, sel, cnt, decode, **kw):
    call = dsa.sparse_attn_decode_fp8 if decode else dsa.sparse_attn_prefill_fp8
    out, lse = call(cache, b.seqs, b.queries, q, sel.cuda(), cnt.cuda(), dev_err=b.err, **kw)
    return out.cpu().double(), lse.cpu().double()


def check_attn(b, host, got, q, sel, cnt, sm_scale=1 / math.sqrt(128)):
    (k, ks), (v, vs) = host
    out, lse, otol, ltol = ref.attention(q.double(), ref.stored(k, ks), ref.stored(v, vs), b.table, b.block, b.seq,
                                         b.pos.tolist(), sel, cnt, sm_scale)
    d = (got[0] - out).abs() - otol
    assert float(d.max()) <= 0, (float(d.max()), float(out.abs().mean()))
    empty = lse == -math.inf
    assert torch.equal(got[1] == -math.inf, empty)
    assert bool(((got[1] - lse).abs() <= ltol)[~empty].all()), float((got[1] - lse).abs()[~empty].max())


@pytest.mark.parametrize("decode", [True, False], ids=["decode_entry", "prefill_entry"])
@pytest.mark.parametrize("name", sorted(ATTN))
def test_attention_fp8(name, decode, cuda_device):
    kw = dict(ATTN[name])
    k = kw.pop("k")
    b = Batch(seed=21, **kw)
    host, cache = b.cache8(nan_slots=True)      # unwritten slots hold NaN codes
    q = torch.randn(b.T, b.hq, 128, generator=b.gen).bfloat16() * 2
    sel, cnt = selection(b, k)
    got = attend(b, cache, q.cuda(), sel, cnt, decode)
    assert int(b.err) == 0
    check_attn(b, host, got, q, sel, cnt)


def test_attention_fp8_rows_without_blocks_and_bad_selections(cuda_device):
    b = Batch((300, 500), (4, 3), 2, 8, seed=22)
    host, cache = b.cache8()
    q = torch.randn(b.T, b.hq, 128, generator=b.gen).bfloat16()
    sel, cnt = selection(b, 4)
    cnt[1] = 0                       # nothing selected
    cnt[3] = 9                       # more than k_max: the row reads as empty
    good = cnt.clone()
    good[3] = 0
    for decode in (True, False):
        b.err.zero_()
        got = attend(b, cache, q.cuda(), sel, cnt, decode)
        check_attn(b, host, got, q, sel, good)
        assert bool((got[0][1] == 0).all()) and bool((got[1][1] == -math.inf).all())
    sel2, cnt2 = sel.clone(), good.clone()
    sel2[5, 0], sel2[6, 1] = 99, -7  # outside the visible blocks: skipped and reported
    keep = [[int(x) for x in sel2[t, :cnt2[t]] if 0 <= x <= int(b.pos[t]) // 64] for t in range(b.T)]
    sel3 = torch.full_like(sel2, -1)
    for t, ids in enumerate(keep):
        sel3[t, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
    cnt3 = torch.tensor([len(i) for i in keep], dtype=torch.int32)
    for decode in (True, False):
        b.err.zero_()
        got = attend(b, cache, q.cuda(), sel2, cnt2, decode)
        assert int(b.err) == _lib.DEV_ERR_SEL
        check_attn(b, host, got, q, sel3, cnt3)
    bad = b.table.clone()
    bad[0, int(sel[0, 0])] = b.pages         # a page outside the pool: skipped and reported
    b.seqs = dsa.SeqBatch(bad.cuda(), b.seqs.seq_lens)
    b.err.zero_()
    attend(b, cache, q.cuda(), sel, good, True)
    assert int(b.err) == _lib.DEV_ERR_PAGE


@pytest.mark.parametrize("lens,n_new,hkv,hq,k", [((300, 500), (4, 3), 2, 8, 4), ((3000,), (1,), 2, 8, 47),
                                                ((200,) * 700, (1,) * 700, 2, 4, 3)],
                         ids=["teams", "split_contexts", "pairs_per_warp"])
def test_attention_fp8_padded_batch(lens, n_new, hkv, hq, k, cuda_device):
    """Queries behind the last sequence's: the others' results as without them, their rows as they were."""
    b = Batch(lens, n_new, hkv, hq, seed=26)
    host, cache = b.cache8()
    q = torch.randn(b.T, b.hq, 128, generator=b.gen).bfloat16()
    sel, cnt = selection(b, k)
    pad = 5
    more = lambda t: torch.cat([t, t[:1].expand(pad, *t.shape[1:])]).contiguous()  # noqa: E731
    queries = dsa.QueryBatch(b.queries.cu_q, more(b.pos).cuda())
    for call, ws in ((dsa.sparse_attn_decode_fp8, True), (dsa.sparse_attn_prefill_fp8, False)):
        want = call(cache, b.seqs, b.queries, q.cuda(), sel.cuda(), cnt.cuda())
        out = torch.full((b.T + pad, b.hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((b.T + pad, b.hq), 7.0, device="cuda")
        kw = dict(workspace=torch.zeros(dsa.decode_workspace_size(b.T + pad, b.hq, b.hkv, k), dtype=torch.uint8,
                                        device="cuda")) if ws else {}
        for _ in range(2):   # the second time on the workspace that the first one leaves
            call(cache, b.seqs, queries, more(q).cuda(), more(sel).cuda(), more(cnt).cuda(), out=out, lse=lse,
                 dev_err=b.err, **kw)
            assert int(b.err) == 0
            assert bool((out[b.T:] == 7).all()) and bool((lse[b.T:] == 7).all())
            # the padding may change how a pair is split, and with it the running maxima that the
            # weights are rounded against: two results differ by their roundings to bf16 and by
            # 2 * 2^-11 of the weighted |v|, which is at most 448 * 2^-5 here; lse by two fp32 sums
            # of at most 3000 terms
            d = (out[:b.T].float() - want[0].float()).abs()
            assert bool((d <= want[0].float().abs() * 2 * BF16_HALF + 2 * 2.0 ** -11 * 448 * 2.0 ** -5).all())
            assert bool(((lse[:b.T] - want[1]).abs() <= 2 * 3008 * 2.0 ** -24).all())


def test_attention_fp8_value_ranges(cuda_device):
    """Scales far apart between tiles, queries from 2^-90 to 2^60, a zero query, large and
    negative logits: within the tolerances of the same definition."""
    b = Batch((640, 640), (3, 3), 1, 8, seed=23)
    host, cache = b.cache8(spread=1)
    (k, ks), (v, vs) = host
    far = torch.exp2(torch.randint(-20, 20, vs.shape, generator=b.gen).float()) * 1.37
    vs.copy_(far)
    ks.mul_(1.21)
    cache.v_scale.copy_(vs)
    cache.k_scale.copy_(ks)
    q = torch.randn(b.T, b.hq, 128, generator=b.gen)
    q[0] *= 2.0 ** -90
    q[1] *= 40
    q[2] = 0
    q[3, :, :64] *= 2.0 ** -40
    q[4, 0] = -q[4, 0].abs()
    q = q.bfloat16()
    sel, cnt = selection(b, 5)
    for decode in (True, False):
        check_attn(b, host, attend(b, cache, q.cuda(), sel, cnt, decode), q, sel, cnt)
        check_attn(b, host, attend(b, cache, q.cuda(), sel, cnt, decode, sm_scale=0.3), q, sel, cnt, 0.3)
    # a very large query with a scale that brings the logits back
    big = (torch.randn(b.T, b.hq, 128, generator=b.gen) * 2.0 ** 60).bfloat16()
    got = attend(b, cache, big.cuda(), sel, cnt, True, sm_scale=2.0 ** -63)
    check_attn(b, host, got, big, sel, cnt, 2.0 ** -63)


def test_attention_fp8_nan_reaches_only_the_rows_that_use_it(cuda_device):
    b = Batch((640,), (4,), 2, 8, seed=24)
    host, cache = b.cache8()
    q = torch.randn(b.T, b.hq, 128, generator=b.gen).bfloat16()
    q[1, 2, 7] = math.nan
    q[2, 5, 9] = math.inf
    sel, cnt = selection(b, 4)
    for decode in (True, False):
        out, lse = attend(b, cache, q.cuda(), sel, cnt, decode)
        bad = torch.zeros(b.T, b.hq, dtype=torch.bool)
        bad[1, 2] = bad[2, 5] = True
        assert torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad)
        assert torch.equal(lse.isnan(), bad)
    # a NaN key in the first selected block of query 0, KV head 1: heads 4..7 of the queries that select it
    blk = int(sel[0, 0])
    cache.k_pool[int(b.table[0, blk]), 3, 1, 50] = 0x7F
    q[1, 2, 7], q[2, 5, 9] = 0.5, 0.25
    for decode in (True, False):
        out, lse = attend(b, cache, q.cuda(), sel, cnt, decode)
        bad = torch.zeros(b.T, b.hq, dtype=torch.bool)
        for t in range(b.T):
            if blk in sel[t].tolist():
                bad[t, 4:] = True
        assert torch.equal(out.isnan().any(-1), bad) and torch.equal(lse.isnan(), bad)


def test_attention_fp8_workspace_is_reusable_and_calls_repeat(cuda_device):
    """The same call twice with one workspace gives the same bits; float8 tensors are taken as codes."""
    b = Batch((3000,), (1,), 2, 8, seed=25)
    host, cache = b.cache8()
    q = torch.randn(1, 8, 128, generator=b.gen).bfloat16().cuda()
    sel, cnt = selection(b, 47)
    ws = torch.zeros(dsa.decode_workspace_size(1, 8, 2, 47), dtype=torch.uint8, device="cuda")
    one = attend(b, cache, q, sel, cnt, True, workspace=ws)
    two = attend(b, cache, q, sel, cnt, True, workspace=ws)
    f8 = dsa.PagedKVCacheFP8(cache.k_pool.view(torch.float8_e4m3fn), cache.v_pool.view(torch.float8_e4m3fn),
                             cache.kc_pool, cache.k_scale, cache.v_scale)
    three = attend(b, f8, q, sel, cnt, True, workspace=ws)
    for other in (two, three):
        assert torch.equal(one[0], other[0]) and torch.equal(one[1], other[1])


def test_pools_past_32_bits(cuda_device):
    """Pools of more than 4 GiB: rows and tiles at the far end are appended to and attended over."""
    pages, hkv = 70000, 8                       # 4.6 GB of codes each for K and V
    pool = [torch.zeros((pages, 64, hkv, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = [torch.zeros((pages, 1, hkv), device="cuda") for _ in range(2)]
    cache = dsa.PagedKVCacheFP8(*pool, torch.zeros((pages, 64), dtype=torch.int8, device="cuda"), *scale)
    g = torch.Generator().manual_seed(41)
    table = torch.tensor([[pages - 1, 5, pages - 2]], dtype=torch.int32, device="cuda")
    x = torch.randn(150, hkv, 128, generator=g).bfloat16()
    y = torch.randn(150, hkv, 128, generator=g).bfloat16()
    seqs = dsa.SeqBatch(table, torch.tensor([150], dtype=torch.int32, device="cuda"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.kv_append_fp8(cache, seqs, torch.tensor([0, 150], dtype=torch.int32, device="cuda"), x.cuda(), y.cuda(),
                      dev_err=err)
    q = torch.randn(1, 8 * hkv, 128, generator=g).bfloat16()
    queries = dsa.QueryBatch(torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                             torch.tensor([149], dtype=torch.int32, device="cuda"))
    sel = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    out, lse = dsa.sparse_attn_decode_fp8(cache, seqs, queries, q.cuda(), sel,
                                          torch.tensor([3], dtype=torch.int32, device="cuda"), dev_err=err)
    assert int(err) == 0
    t = table[0].long()
    small = [ref.stored(p[t].cpu(), s[t].cpu()) for p, s in zip(pool, scale)]
    for got, want in zip(small, (x, y)):
        d = (got.reshape(192, hkv, 128)[:150] - want.double()).abs()
        step = want.double().abs() * E4M3_HALF + 2.0 ** -10 * 2.0 ** -5      # scales are at most 2^-5: |x| < 14
        assert bool((d <= step).all())
    w, wl, otol, ltol = ref.attention(q.double(), *small, torch.tensor([[0, 1, 2]]), 64, [0], [149], sel.cpu(), [3],
                                      1 / math.sqrt(128))
    assert bool(((out.cpu().double() - w).abs() <= otol).all()) and bool(((lse.cpu().double() - wl).abs() <= ltol).all())
    assert not bool(pool[0][6].any())


# ----------------------------------------------------------------------------- together

def test_attention_right_behind_the_append(cuda_device):
    """The attention reads the queries, codes and scales of the append launched just before it
    (it may start early): eager and replayed from a graph, many times, always the same bits."""
    b = Batch((2000, 900, 70), (300, 1, 70), 2, 16, seed=33)
    _, _, rope = rotary()
    host, cache = b.cache8()
    sel, cnt = selection(b, 6)
    sel, cnt, kc = sel.cuda(), cnt.cuda(), b.kc.cuda()
    state = (cache.k_pool, cache.v_pool, cache.kc_pool, cache.k_scale, cache.v_scale)
    start = [t.clone() for t in state]
    q_rot, out = torch.empty_like(b.dq), torch.empty_like(b.dq)
    lse = torch.empty((b.T, b.hq), device="cuda")
    ws = torch.zeros(dsa.decode_workspace_size(b.T, b.hq, b.hkv, 6), dtype=torch.uint8, device="cuda")

    def both(decode):
        dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q, b.dk, b.dv, kc, rope, queries=b.queries, q=b.dq, q_out=q_rot,
                          dev_err=b.err)
        if decode:
            dsa.sparse_attn_decode_fp8(cache, b.seqs, b.queries, q_rot, sel, cnt, out=out, lse=lse, workspace=ws,
                                       dev_err=b.err)
        else:
            dsa.sparse_attn_prefill_fp8(cache, b.seqs, b.queries, q_rot, sel, cnt, out=out, lse=lse, dev_err=b.err)

    def restore():
        for t, old in zip(state, start):
            t.copy_(old)
        q_rot.zero_()
        out.zero_()
        torch.cuda.synchronize()

    for decode in (True, False):
        restore()
        both(decode)
        torch.cuda.synchronize()
        want = out.clone(), lse.clone()
        few = torch.tensor([0, 150, 299, 300, 301, 370])
        (k, ks), (v, vs) = ((cache.k_pool, cache.k_scale), (cache.v_pool, cache.v_scale))
        w, wl, otol, _ = ref.attention(q_rot.cpu()[few].double(), ref.stored(k.cpu(), ks.cpu()),
                                       ref.stored(v.cpu(), vs.cpu()), b.table, b.block, [b.seq[i] for i in few],
                                       b.pos[few].tolist(), sel.cpu()[few], cnt.cpu()[few], 1 / math.sqrt(128))
        assert bool(((out.cpu()[few].double() - w).abs() <= otol).all())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both(decode)
        for i in range(20):
            restore()
            graph.replay() if i % 2 else both(decode)
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert int(b.err) == 0


def test_two_batches_on_two_streams(cuda_device):
    """Independent batches in flight on streams of their own, outputs allocated by the calls:
    the results of each alone."""
    batches = []
    for i in range(2):
        b = Batch((3000, 500 + i), (1, 1), 2, 16, seed=50 + i)
        host, cache = b.cache8()
        sel, cnt = selection(b, 8)
        batches.append((b, cache, torch.randn(b.T, b.hq, 128, generator=b.gen).bfloat16().cuda(), sel.cuda(), cnt.cuda()))
    _, _, rope = rotary()

    def work(b, cache, q, sel, cnt, stream=None):
        r = dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q, b.dk, b.dv, None, rope, queries=b.queries, q=q,
                              stream=stream)
        return r, dsa.sparse_attn_decode_fp8(cache, b.seqs, b.queries, r, sel, cnt, stream=stream)

    alone = []
    for a in batches:
        r, (out, lse) = work(*a)
        torch.cuda.synchronize()
        alone.append((r.clone(), out.clone(), lse.clone()))
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    kept = []
    for _ in range(20):
        for a, s in zip(batches, streams):
            kept.append(work(*a, stream=s))
    torch.cuda.synchronize()
    for i, (r, (out, lse)) in enumerate(kept):
        want = alone[i % 2]
        assert torch.equal(r, want[0]) and torch.equal(out, want[1]) and torch.equal(lse, want[2])


def test_calls_without_the_native_reader(cuda_device, monkeypatch):
    """The binding's own marshalling makes the same calls as the native reader's."""
    got = []
    for native in (True, False):
        if not native:
            monkeypatch.setattr(dsa, "_native", None)
        b, rope, pos, _ = make("three_axes", seed=61)
        _, cache = b.cache8()
        q = dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q, b.dk, b.dv, b.kc.cuda(), rope, pos_new=pos, queries=b.queries,
                              q=b.dq, pos_q=pos, dev_err=b.err)
        (_, _), c16 = b.cache16()
        q16 = dsa.kv_append_rope(c16, b.seqs, b.queries.cu_q, b.dk, b.dv, None, rope, pos_new=pos, queries=b.queries,
                                 q=b.dq, pos_q=pos, dev_err=b.err)
        sel, cnt = selection(b, 3)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        ws = torch.zeros(dsa.decode_workspace_size(b.T, b.hq, b.hkv, 3), dtype=torch.uint8, device="cuda")
        dsa.sparse_attn_decode_fp8(cache, b.seqs, b.queries, q, sel.cuda(), cnt.cuda(), out=out, lse=lse, workspace=ws,
                                   dev_err=b.err)
        out2, lse2 = dsa.sparse_attn_prefill_fp8(cache, b.seqs, b.queries, q, sel.cuda(), cnt.cuda(),
                                                 out=torch.empty_like(out), lse=torch.empty_like(lse))
        assert int(b.err) == 0
        got.append([t.cpu().view(torch.uint8) for t in (q, q16, out, lse, out2, lse2, cache.k_pool, cache.v_pool,
                                                        cache.k_scale, cache.v_scale, cache.kc_pool, c16.k_pool)])
    for x, y in zip(*got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("native", [True, False], ids=["native", "python"])
def test_binding_refuses_what_would_read_out_of_bounds(native, cuda_device, monkeypatch):
    if not native:
        monkeypatch.setattr(dsa, "_native", None)
    b = Batch((70, 90), (3, 1), 2, 4, seed=60)
    _, cache = b.cache8()
    _, _, rope = rotary()
    sel, cnt = selection(b, 2)
    q = b.dq
    short = dsa.QueryBatch(b.queries.cu_q[:2].clone(), b.queries.q_pos)
    with pytest.raises(ValueError, match="cu_q"):
        dsa.sparse_attn_decode_fp8(cache, b.seqs, short, q, sel.cuda(), cnt.cuda())
    with pytest.raises(ValueError, match="k_max"):
        dsa.sparse_attn_decode_fp8(cache, b.seqs, b.queries, q, sel[:2].cuda(), cnt.cuda())
    with pytest.raises(ValueError, match="lse"):
        dsa.sparse_attn_decode_fp8(cache, b.seqs, b.queries, q, sel.cuda(), cnt.cuda(), lse=torch.empty(1, 4, device="cuda"))
    with pytest.raises(ValueError, match="must be"):
        dsa.sparse_attn_decode_fp8(cache, b.seqs, b.queries, q.half(), sel.cuda(), cnt.cuda())
    with pytest.raises(ValueError, match="v_new"):
        dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q, b.dk, b.dv[:2])
    with pytest.raises(ValueError, match="cu_new"):
        dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q[:2].clone(), b.dk, b.dv)
    with pytest.raises(ValueError, match="needs v_new"):
        dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q, b.dk, None)
    with pytest.raises(ValueError, match="contiguous"):
        dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q, b.dk.transpose(1, 2).contiguous().transpose(1, 2), b.dv)
    with pytest.raises(ValueError, match="pos_new"):
        dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q, b.dk, b.dv, None, rope, pos_new=b.queries.q_pos[:2])
    with pytest.raises(ValueError, match="q_out"):
        dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q, b.dk, b.dv, None, rope, queries=b.queries, q=q,
                          q_out=q[:, :2].contiguous())
    with pytest.raises(ValueError, match="CUDA tensors only"):
        dsa.kv_append_fp8(cache, b.seqs, b.queries.cu_q, b.dk.cpu(), b.dv)
    with pytest.raises(TypeError):
        dsa.sparse_attn_decode(cache, b.seqs, b.queries, q, sel.cuda(), cnt.cuda())
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = torch.zeros(dsa.decode_workspace_size(b.T, b.hq, b.hkv, 2), dtype=torch.uint8, device="cuda")
    kw = dict(out=out, lse=lse, workspace=ws)
    for bad in (dict(workspace=ws[:64]), dict(sm_scale=-1.0)):
        with pytest.raises(dsa.DsaError):
            dsa.sparse_attn_decode_fp8(cache, b.seqs, b.queries, q, sel.cuda(), cnt.cuda(), **{**kw, **bad})
    for bad in (dict(out=out.view(b.T, -1)), dict(lse=lse[:2].contiguous()), dict(out=out.float()),
                dict(dev_err=b.err.long())):
        with pytest.raises(ValueError):
            dsa.sparse_attn_decode_fp8(cache, b.seqs, b.queries, q, sel.cuda(), cnt.cuda(), **{**kw, **bad})
    with pytest.raises(ValueError, match="cu_q"):
        dsa.sparse_attn_decode_fp8(cache, b.seqs, short, q, sel.cuda(), cnt.cuda(), **kw)
    with pytest.raises(ValueError, match="k_max"):
        dsa.sparse_attn_decode_fp8(cache, b.seqs, b.queries, q, sel[:2].cuda(), cnt.cuda(), **kw)
    with pytest.raises(ValueError, match="seq_lens"):
        dsa.sparse_attn_decode_fp8(cache, dsa.SeqBatch(b.seqs.block_table, b.seqs.seq_lens[:1]), b.queries, q, sel.cuda(),
                                   cnt.cuda(), **kw)
    small = dsa.PagedKVCacheFP8(cache.k_pool, cache.v_pool[:1], cache.kc_pool, cache.k_scale, cache.v_scale)
    with pytest.raises(ValueError, match="differ in shape"):
        dsa.sparse_attn_decode_fp8(small, b.seqs, b.queries, q, sel.cuda(), cnt.cuda(), **kw)
    with pytest.raises(ValueError, match="differ in shape"):
        dsa.kv_append_fp8(small, b.seqs, b.queries.cu_q, b.dk, b.dv)
    few = dsa.PagedKVCacheFP8(cache.k_pool, cache.v_pool, cache.kc_pool, cache.k_scale[:1], cache.v_scale)
    with pytest.raises(ValueError, match="k_scale"):
        dsa.kv_append_fp8(few, b.seqs, b.queries.cu_q, b.dk, b.dv)



@pytest.mark.parametrize("decode,fused", [(True, False), (True, True), (False, True), (False, False)],
                         ids=["decode", "decode_fused_select", "prefill_fused_select", "prefill"])
@pytest.mark.parametrize("fp8", [True, False], ids=["fp8", "bf16"])
def test_step_with_rotation(fp8, decode, fused, cuda_device):
    """append (rotated) -> select -> attention through step() and PreparedStep: the selection is
    that of an append without rotation, the attention that of the definition over what the append
    stored; replayed from a CUDA graph it gives the same bits."""
    n_new = (1, 1, 1) if decode else (40, 1, 90)
    b = Batch((900, 300, 1700), n_new, 2, 8, seed=31, packed=True)
    inv, _, rope = rotary()
    host, cache = b.cache8() if fp8 else b.cache16()
    q_idx = torch.randint(-127, 128, (b.T, 8, 64), generator=b.gen, dtype=torch.int8).cuda()
    w = torch.randint(0, 17, (b.T, 8), generator=b.gen, dtype=torch.int32).cuda()
    kps = torch.tensor([5, 3, 6], dtype=torch.int32).cuda()
    args = dict(k_new=b.dk, v_new=b.dv, kc_new=b.kc.cuda(), q=b.dq, q_idx=q_idx, w=w, k_per_seq=kps, k_max=6,
                decode=decode, fused_select=fused, rope=rope, dev_err=b.err)
    start = [t.clone() for t in (cache.k_pool, cache.v_pool, cache.kc_pool)]
    scales = [t.clone() for t in (cache.k_scale, cache.v_scale)] if fp8 else []
    bufs = dsa.step(cache, b.seqs, b.queries, **args)
    torch.cuda.synchronize()
    assert int(b.err) == 0
    kw, ks = ref.rotate(b.k.double(), b.pos[None], inv)
    if fp8:
        check_fp8_append(b, host, cache, kw, ks)
    q_rot = bufs["q_rot"].cpu()
    want, slack = ref.rotate(b.q.double(), b.pos[None], inv)
    check_rows(q_rot, want, slack, BF16_HALF)
    sel, cnt = bufs["sel"].cpu(), bufs["cnt"].cpu()
    plain = dsa.PagedKVCache(torch.zeros(b.shape(), dtype=torch.bfloat16, device="cuda"),
                             torch.zeros(b.shape(), dtype=torch.bfloat16, device="cuda"), cache.kc_pool)
    sel0, cnt0 = dsa.select_blocks(plain, b.seqs, b.queries, q_idx, w, kps, 6)
    assert torch.equal(sel0.cpu(), sel) and torch.equal(cnt0.cpu(), cnt)
    if fp8:
        k, v = ref.stored(cache.k_pool.cpu(), cache.k_scale.cpu()), ref.stored(cache.v_pool.cpu(), cache.v_scale.cpu())
    else:
        k, v = cache.k_pool.cpu().double(), cache.v_pool.cpu().double()
    few = torch.randperm(b.T, generator=b.gen)[:24].sort().values if b.T > 24 else torch.arange(b.T)
    out, lse, otol, ltol = ref.attention(q_rot[few].double(), k, v, b.table, b.block, [b.seq[i] for i in few],
                                         b.pos[few].tolist(), sel[few], cnt[few], 1 / math.sqrt(128),
                                         2.0 ** -11 if fp8 else BF16_HALF)
    assert bool(((bufs["out"].cpu()[few].double() - out).abs() <= otol).all())
    assert bool(((bufs["lse"].cpu()[few].double() - lse).abs() <= ltol).all())
    first = {n: bufs[n].clone() for n in ("out", "lse", "sel", "q_rot")}
    after = [t.clone() for t in (cache.k_pool, cache.v_pool, cache.kc_pool)]

    def restore():
        for t, old in zip((cache.k_pool, cache.v_pool, cache.kc_pool), start):
            t.copy_(old)
        for t, old in zip((cache.k_scale, cache.v_scale) if fp8 else (), scales):
            t.copy_(old)
        for n in first:
            bufs[n].fill_(0)

    def same():
        torch.cuda.synchronize()
        for n, t in first.items():
            assert torch.equal(bufs[n], t), n
        for t, old in zip((cache.k_pool, cache.v_pool, cache.kc_pool), after):
            assert torch.equal(t.view(torch.uint8), old.view(torch.uint8))

    prepared = dsa.PreparedStep(cache, b.seqs, b.queries, bufs=bufs, **args)
    restore()
    prepared()
    same()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        prepared(stream=torch.cuda.current_stream())
    for _ in range(2):
        restore()
        torch.cuda.synchronize()
        graph.replay()
        same()
