"""One workspace through calls of different batches: zero-filled once, it serves
every later call, whatever the batch size, the heads per KV head and (for the
attention) the cache's type.  Each call's results are the bits of the same call
on a fresh workspace; the kernels merge in a fixed order."""
import pytest
import torch

import dynamic_block_sparse_dsa_b200 as dsa

from test_gpu_rope_fp8 import Batch, selection

pytestmark = pytest.mark.gpu


def _decode_call(T, hkv, group, k, fp8, seed):
    """(call(workspace) -> (out, lse), workspace size) of a decode batch of T contexts."""
    b = Batch(tuple(1500 + 61 * i for i in range(T)), (1,) * T, hkv, hkv * group, seed=seed)
    cache = (b.cache8() if fp8 else b.cache16())[1]
    q = torch.randn(T, hkv * group, 128, generator=b.gen).bfloat16().cuda()
    sel, cnt = selection(b, k)
    sel, cnt = sel.cuda(), cnt.cuda()
    fn = dsa.sparse_attn_decode_fp8 if fp8 else dsa.sparse_attn_decode

    def call(ws):
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        fn(cache, b.seqs, b.queries, q, sel, cnt, out=out, lse=lse, workspace=ws, dev_err=b.err)
        assert int(b.err) == 0
        return out, lse

    return call, dsa.decode_workspace_size(T, hkv * group, hkv, k)


# batches of 2 to 320 pairs (split over CTAs below half as many pairs as SMs in the 8-bit kernel,
# at any unaligned boundary in the bf16 one), growing, shrinking and growing again
ORDERS = {
    "fp8": [(8, 8, 8, True), (9, 8, 8, True), (8, 8, 8, True), (9, 8, 8, True)],
    "bf16": [(20, 8, 8, False), (40, 8, 8, False), (20, 8, 8, False), (40, 8, 8, False)],
    "mixed": [(20, 8, 4, False), (9, 8, 4, True), (2, 1, 4, True), (40, 8, 4, False), (9, 8, 4, True), (3, 1, 4, False),
              (40, 8, 4, False)],
    "groups": [(4, 2, 16, True), (9, 8, 1, True), (40, 8, 1, False), (4, 2, 16, False), (9, 8, 8, True), (40, 8, 4, False),
               (9, 8, 1, True)],
}


@pytest.mark.parametrize("order", sorted(ORDERS))
def test_decode_workspace_serves_batches_of_any_size(order, cuda_device):
    calls, need = {}, 0
    for i, key in enumerate(ORDERS[order]):
        if key not in calls:
            T, hkv, group, fp8 = key
            call, size = _decode_call(T, hkv, group, 16, fp8, seed=70 + i)
            want = call(torch.zeros(size, dtype=torch.uint8, device="cuda"))
            assert not bool((want[0] == 7).all(-1).any())      # every row written
            calls[key] = call, want
            need = max(need, size)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for n, key in enumerate(ORDERS[order]):
        call, want = calls[key]
        out, lse = call(ws)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), (order, n, key)


def _select_case(T, blocks=20000, seed=5):
    """A decode batch whose contexts share their pages (only the coarse keys are read): several
    chunks of candidates per query."""
    g = torch.Generator().manual_seed(seed + T)
    pages = blocks
    pool = torch.zeros((pages, 64, 1, 128), dtype=torch.uint8, device="cuda")
    scale = torch.ones((pages, 1, 1), device="cuda")
    kc = torch.randint(-127, 128, (pages, 64), generator=torch.Generator().manual_seed(seed), dtype=torch.int8).cuda()
    cache = dsa.PagedKVCacheFP8(pool, pool, kc, scale, scale)
    table = torch.randperm(pages, generator=g).int()[None].expand(T, pages).contiguous().cuda()
    lens = torch.full((T,), blocks * 64, dtype=torch.int32).cuda()
    cu = torch.arange(T + 1, dtype=torch.int32).cuda()
    q_idx = torch.randint(-127, 128, (T, 16, 64), generator=g, dtype=torch.int8).cuda()
    w = torch.randint(0, 17, (T, 16), generator=g, dtype=torch.int32).cuda()
    kps = torch.full((T,), 64, dtype=torch.int32).cuda()
    seqs, queries = dsa.SeqBatch(table, lens), dsa.QueryBatch(cu, lens - 1)

    def call(ws):
        sel = torch.full((T, 64), -9, dtype=torch.int32, device="cuda")
        cnt = torch.full((T,), -9, dtype=torch.int32, device="cuda")
        return dsa.select_blocks(cache, seqs, queries, q_idx, w, kps, 64, sel=sel, cnt=cnt, workspace=ws)
    return call


def test_select_workspace_serves_batches_of_any_size(cuda_device):
    sizes = (8, 100, 3, 100, 40, 8, 100)
    calls = {}
    for T in set(sizes):
        call = _select_case(T)
        want = call(torch.zeros(dsa.select_workspace_size(T), dtype=torch.uint8, device="cuda"))
        assert bool((want[1] == 64).all())
        calls[T] = call, want
    ws = torch.zeros(dsa.select_workspace_size(max(sizes)), dtype=torch.uint8, device="cuda")
    for n, T in enumerate(sizes):
        call, want = calls[T]
        sel, cnt = call(ws)
        assert torch.equal(sel, want[0]) and torch.equal(cnt, want[1]), (n, T)


def _fused_call(T, hkv, group, seed):
    """A decode batch through the single-launch step; the appended rows are the same every time."""
    b = Batch(tuple(5000 + 777 * i for i in range(T)), (1,) * T, hkv, hkv * group, seed=seed)
    cache = b.cache16()[1]
    q_idx = torch.randint(-127, 128, (T, 16, 64), generator=b.gen, dtype=torch.int8).cuda()
    w = torch.randint(0, 17, (T, 16), generator=b.gen, dtype=torch.int32).cuda()
    kps = torch.full((T,), 12, dtype=torch.int32).cuda()
    kc = b.kc.cuda()

    def call(ws):
        got = [torch.full((T, 12), -9, dtype=torch.int32, device="cuda"), torch.full((T,), -9, dtype=torch.int32, device="cuda"),
               torch.full_like(b.dq, 7.0), torch.full(b.dq.shape[:2], 7.0, device="cuda")]
        dsa.decode_fused(cache, b.seqs, b.queries, b.queries.cu_q, b.dk, b.dv, kc, q_idx, w, kps, 12, b.dq, sel=got[0],
                         cnt=got[1], out=got[2], lse=got[3], workspace=ws, dev_err=b.err)
        assert int(b.err) == 0
        return got

    return call, dsa.decode_fused_workspace_size(T, hkv * group, hkv, 12)


def test_fused_decode_workspace_serves_batches_of_any_size(cuda_device):
    order = [(3, 2, 4), (40, 2, 4), (3, 2, 4), (2, 1, 16), (40, 2, 4), (17, 8, 2), (2, 1, 16), (40, 2, 4)]
    calls, need = {}, 0
    for i, key in enumerate(order):
        if key not in calls:
            call, size = _fused_call(*key, seed=75 + i)
            calls[key] = call, call(torch.zeros(size, dtype=torch.uint8, device="cuda"))
            need = max(need, size)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for n, key in enumerate(order):
        call, want = calls[key]
        for got, w in zip(call(ws), want):
            assert torch.equal(got, w), (n, key)


def test_captured_calls_of_several_batches_share_a_workspace(cuda_device):
    """Graphs of differently sized batches over both caches, captured on one workspace and replayed
    in turn with an eager call among them."""
    keys = [(8, 8, 8, True), (9, 8, 8, True), (40, 8, 8, False), (3, 1, 16, True)]
    cases, need = [], 0
    for i, (T, hkv, group, fp8) in enumerate(keys):
        b = Batch(tuple(1500 + 61 * j for j in range(T)), (1,) * T, hkv, hkv * group, seed=110 + i)
        cache = (b.cache8() if fp8 else b.cache16())[1]
        q = torch.randn(T, hkv * group, 128, generator=b.gen).bfloat16().cuda()
        sel, cnt = (t.cuda() for t in selection(b, 16))
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        fn = dsa.sparse_attn_decode_fp8 if fp8 else dsa.sparse_attn_decode
        size = dsa.decode_workspace_size(T, hkv * group, hkv, 16)

        def call(ws, fn=fn, b=b, cache=cache, q=q, sel=sel, cnt=cnt, out=out, lse=lse):
            fn(cache, b.seqs, b.queries, q, sel, cnt, out=out, lse=lse, workspace=ws, dev_err=b.err)

        call(torch.zeros(size, dtype=torch.uint8, device="cuda"))
        cases.append((call, out, lse, out.clone(), lse.clone(), b.err))
        need = max(need, size)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs = []
    for call, *_ in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(ws)
    for n, i in enumerate((0, 1, 2, 0, 3, 1, 2, 3, 1, 0, 2)):
        call, out, lse, want, want_lse, err = cases[i]
        out.fill_(7)
        lse.fill_(7)
        call(ws) if n % 4 == 3 else graphs[i].replay()
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and int(err) == 0, (n, i)
