"""8-bit attention where a warp takes whole (query, KV head) pairs: batches of
as many pairs as the GPU has warps, and more, with every query checked.

The kernel gives floor(pairs / W) rounds of one pair per warp (W warps on the
GPU: 12 per SM, 8 for more than 8 heads per KV head) and the pairs left over to
teams of a CTA's warps.  The sizes here are derived from the SM count, so that
each case keeps reaching the part of the schedule that its name says."""
import math

import pytest
import torch

import dynamic_block_sparse_dsa_b200 as dsa
from dynamic_block_sparse_dsa_b200 import _lib

import rope_fp8_reference as ref
from test_gpu_rope_fp8 import Batch

pytestmark = pytest.mark.gpu


def definition(b, cache, q, sel, cnt, sm_scale):
    """ref.attention with its tolerances for all queries at once, in float64 on the GPU."""
    k, v = (ref.decode_e4m3(p) * s.double().repeat_interleave(64, dim=1)[..., None]
            for p, s in ((cache.k_pool, cache.k_scale), (cache.v_pool, cache.v_scale)))
    T, hq, _ = q.shape
    hkv, kmax = b.hkv, sel.shape[1]
    group, step = hq // hkv, max(1, (1 << 25) // (kmax * b.block * hkv * 128))
    seq, pos = torch.tensor(b.seq).cuda(), b.pos.cuda().long()
    slot = torch.arange(kmax, device="cuda")
    got = [[], [], [], []]
    for lo in range(0, T, step):
        r = slice(lo, min(lo + step, T))
        ids = sel[r].long()
        used = (slot[None] < cnt[r, None]) & (ids >= 0)
        page = torch.where(used, b.seqs.block_table[seq[r, None], ids.clamp(min=0)].long(), 0)
        tok = ids[..., None] * b.block + torch.arange(b.block, device="cuda")
        seen = (used[..., None] & (tok <= pos[r, None, None])).flatten(1)[:, None, None]      # [t][1][1][n]
        kk, vv = (torch.where(seen[:, 0, 0, :, None, None], x[page].flatten(1, 2), 0.0).transpose(1, 2) for x in (k, v))
        qq = q[r].double().view(-1, hkv, group, 128)
        s = (qq @ kk.transpose(2, 3) * sm_scale).masked_fill(~seen, -math.inf)
        top = s.amax(-1, keepdim=True)
        w = torch.where(seen, (s - top).exp(), 0.0)
        norm = w.sum(-1, keepdim=True)
        some = norm > 0
        p = torch.where(some, w / norm, 0.0)
        out = p @ vv
        n = seen.sum(-1, keepdim=True)
        delta = (qq.abs() @ kk.abs().transpose(2, 3)).amax(-1, keepdim=True) * sm_scale * 140 * 2.0 ** -24 + 2.0 ** -21
        delta = delta + kk.abs().sum(3).amax(-1)[:, :, None, None] * qq.abs().amax(-1, keepdim=True) * sm_scale * 2.0 ** -39
        tiny = torch.where(some, 2.0 ** -25 / norm, 0.0) * vv.abs().sum(2, keepdim=True)
        got[0].append(out.reshape(-1, hq, 128))
        got[1].append(torch.where(some, top + norm.log(), -math.inf).reshape(-1, hq))
        got[2].append((out.abs() * 2.0 ** -8 + (p @ vv.abs()) * (2 * delta + 2.0 ** -11 + n * 2.0 ** -24) + tiny
                       + 1e-30).reshape(-1, hq, 128))
        got[3].append((delta + (n + 8) * 2.0 ** -24).reshape(-1, hq) + got[1][-1].abs() * 2.0 ** -22)
    return [torch.cat(x) for x in got]


def warps(group):
    return torch.cuda.get_device_properties(0).multi_processor_count * (12 if group <= 8 else 8)


# pairs as a function of the warps W; hkv, heads per KV head, k_max, block
CASES = {
    "one_round_exactly": (lambda W: W, 1, 5, 3, 64),
    "one_round_and_teams_of_3": (lambda W: W + 8, 2, 8, 3, 64),
    "one_round_and_teams_of_6": (lambda W: W + 9, 1, 4, 7, 64),
    "one_round_and_whole_ctas": (lambda W: W + 7, 1, 1, 13, 64),
    "two_rounds_and_teams_of_2": (lambda W: 2 * W + W // 3 + 6, 2, 2, 4, 64),
    "two_rounds_and_most_of_a_third": (lambda W: 2 * W + W // 2 + 10, 2, 3, 3, 64),
    "pages_of_256": (lambda W: W + 6, 2, 8, 2, 256),
    "sixteen_heads": (lambda W: 2 * W + 4, 2, 16, 3, 64),
    "eleven_heads_exactly": (lambda W: 2 * W, 2, 11, 2, 64),
    "nine_heads_and_whole_ctas": (lambda W: W + 5, 1, 9, 9, 64),
}


@pytest.mark.parametrize("decode", [True, False], ids=["decode_entry", "prefill_entry"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_attention_fp8_pairs_per_warp(name, decode, cuda_device):
    """Every row of the batch against the definition: rows without blocks, unsorted and partly
    invalid selections, NaN codes in the slots behind each position, queries behind the last
    sequence (left as they were)."""
    of, hkv, group, k, block = CASES[name]
    T = of(warps(group)) // hkv
    # chunks of 1 to 90 queries at the end of contexts of up to 14 blocks
    n_new, lens, left, i = [], [], T, 0
    while left:
        n = min(left, 1 + 37 * i % 90)
        n_new.append(n)
        lens.append(max(n, 1 + 131 * (i + 3) % (14 * block)))
        left -= n
        i += 1
    b = Batch(lens, n_new, hkv, hkv * group, block=block, seed=80)
    _, cache = b.cache8(nan_slots=True)
    q = torch.randn(T, hkv * group, 128, generator=b.gen).bfloat16().cuda()
    sel = torch.full((T, k), -1, dtype=torch.int32)
    cnt = torch.zeros(T, dtype=torch.int32)
    for t in range(T):
        last = int(b.pos[t]) // block
        ids = torch.randperm(last, generator=b.gen)[:k - 1].tolist() + [last]
        sel[t, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
        cnt[t] = len(ids)
    cnt[::53] = 0                        # nothing selected
    cnt[31::97] = k + 1                  # more than k_max: the row reads as empty
    want_cnt = cnt.clone()
    want_cnt[31::97] = 0
    want_sel = sel.clone()
    sel[17::41, 0] = 1 << 20             # outside the visible blocks: skipped
    want_sel[17::41, 0] = -1
    sel, cnt, want_sel, want_cnt = (t.cuda() for t in (sel, cnt, want_sel, want_cnt))
    scale = 1 / math.sqrt(128)
    pad = 3
    more = lambda t: torch.cat([t, t[:1].expand(pad, *t.shape[1:])]).contiguous()  # noqa: E731
    queries = dsa.QueryBatch(b.queries.cu_q, more(b.queries.q_pos))
    for padded in (False, True):
        n = T + (pad if padded else 0)
        grow = more if padded else (lambda t: t)
        out = torch.full((n, hkv * group, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n, hkv * group), 7.0, device="cuda")
        kw = dict(workspace=torch.zeros(dsa.decode_workspace_size(n, hkv * group, hkv, k), dtype=torch.uint8,
                                        device="cuda")) if decode else {}
        b.err.zero_()
        (dsa.sparse_attn_decode_fp8 if decode else dsa.sparse_attn_prefill_fp8)(
            cache, b.seqs, queries if padded else b.queries, grow(q), grow(sel), grow(cnt), out=out, lse=lse,
            dev_err=b.err, **kw)
        assert int(b.err) == _lib.DEV_ERR_SEL
        assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all())
        w, wl, otol, ltol = definition(b, cache, q, want_sel, want_cnt, scale)
        over = (out[:T].double() - w).abs() - otol
        assert float(over.max()) <= 0, (float(over.max()), divmod(int(over.argmax()), 128 * hkv * group))
        empty = wl == -math.inf
        assert torch.equal(lse[:T] == -math.inf, empty) and bool(empty.any())
        assert bool(((lse[:T] - wl).abs() <= ltol)[~empty].all())


@pytest.mark.parametrize("group", [4, 16])
def test_attention_fp8_nan_with_pairs_per_warp(group, cuda_device):
    """A NaN key in one block and a NaN query row, two pairs a warp: only the rows that use them."""
    T = 2 * warps(group) + 5
    b = Batch((640,) * (T // 100 + 1), (100,) * (T // 100) + (T % 100,), 1, group, seed=81)
    _, cache = b.cache8()
    q = torch.randn(T, group, 128, generator=b.gen).bfloat16()
    sel = torch.randint(0, 4, (T, 2), generator=b.gen, dtype=torch.int32)
    sel[:, 1] += 4
    cache.k_pool[int(b.table[1, 2]), 3, 0, 50] = 0x7F
    rows = [1, 250, T - 1]
    bad = torch.zeros(T, group, dtype=torch.bool)
    for t in range(T):
        bad[t] = b.seq[t] == 1 and int(sel[t, 0]) == 2
    for t in rows:
        q[t, group - 1, 7] = math.nan
        bad[t, group - 1] = True
    assert 0 < int(bad.sum()) < bad.numel() // 4
    cnt = torch.full((T,), 2, dtype=torch.int32)
    for call in (dsa.sparse_attn_decode_fp8, dsa.sparse_attn_prefill_fp8):
        out, lse = call(cache, b.seqs, b.queries, q.cuda(), sel.cuda(), cnt.cuda(), dev_err=b.err)
        assert int(b.err) == 0
        assert torch.equal(out.isnan().all(-1).cpu(), bad) and torch.equal(out.isnan().any(-1).cpu(), bad)
        assert torch.equal(lse.isnan().cpu(), bad)
