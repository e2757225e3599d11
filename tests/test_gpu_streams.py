"""Calls on a stream of their own while the current stream is busy: what a call
allocates (workspaces with their zero fill above all) is ordered on its stream."""
import pytest
import torch

import dynamic_block_sparse_dsa_b200 as dsa

from test_gpu_rope_fp8 import Batch, rotary, selection

pytestmark = pytest.mark.gpu

BUSY = 400_000_000   # cycles: about 0.2 s


def _step_case(fp8, fused_decode=False, seed=100):
    b = Batch((9000, 500, 70), (1, 1, 1), 2, 16, seed=seed)
    host, cache = b.cache8() if fp8 else b.cache16()
    q_idx = torch.randint(-127, 128, (b.T, 16, 64), generator=b.gen, dtype=torch.int8).cuda()
    w = torch.randint(0, 17, (b.T, 16), generator=b.gen, dtype=torch.int32).cuda()
    kps = torch.tensor([16, 7, 2], dtype=torch.int32).cuda()
    args = dict(k_new=b.dk, v_new=b.dv, kc_new=b.kc.cuda(), q=b.dq, q_idx=q_idx, w=w, k_per_seq=kps, k_max=16, dev_err=b.err)
    if fused_decode:
        args["fused_decode"] = True
    else:
        args.update(fused_select=True, rope=rotary()[2])
    return b, cache, args


def _dirty(n=64):
    """Memory that the allocator hands out again is not zero."""
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            del_me = [torch.full((1 << 20,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(n)]
            del del_me
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["fp8_rope", "bf16_rope", "fused_decode"])
def test_first_step_on_a_side_stream(kind, cuda_device):
    """step() allocates its buffers: the same results as on an idle device, although the current
    stream has 0.2 s of work ahead of anything issued on it."""
    b, cache, args = _step_case(kind == "fp8_rope", kind == "fused_decode")
    want = {k: v.clone() for k, v in dsa.step(cache, b.seqs, b.queries, **args).items()}
    side = torch.cuda.Stream()
    for i in range(3):
        _dirty()
        if i != 1:
            torch.cuda._sleep(BUSY)
        got = dsa.step(cache, b.seqs, b.queries, stream=side, **args)
        side.synchronize()
        for n in ("sel", "cnt", "out", "lse") + (("q_rot",) if "q_rot" in want else ()):
            assert torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)), (kind, i, n)
        torch.cuda.synchronize()
    assert int(b.err) == 0


def test_prepared_step_is_ready_on_any_stream(cuda_device):
    """A PreparedStep that allocated its buffers behind a busy current stream, called on another."""
    b, cache, args = _step_case(True)
    want = {k: v.clone() for k, v in dsa.step(cache, b.seqs, b.queries, **args).items()}
    side = torch.cuda.Stream()
    for given in (None, side):
        _dirty()
        torch.cuda._sleep(BUSY)
        ps = dsa.PreparedStep(cache, b.seqs, b.queries, stream=given, **args)
        got = ps() if given is not None else ps(stream=side)
        side.synchronize()
        for n in ("sel", "cnt", "out", "lse", "q_rot"):
            assert torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)), n
        torch.cuda.synchronize()
    assert int(b.err) == 0


def test_single_calls_on_a_side_stream(cuda_device):
    """The calls that allocate their own outputs and workspaces, each behind a busy current stream."""
    b = Batch((3000,), (1,), 2, 8, seed=101)
    _, c8 = b.cache8()
    _, c16 = b.cache16()
    q = torch.randn(1, 8, 128, generator=b.gen).bfloat16().cuda()
    sel, cnt = selection(b, 47)
    sel, cnt = sel.cuda(), cnt.cuda()
    q_idx = torch.randint(-127, 128, (1, 16, 64), generator=b.gen, dtype=torch.int8).cuda()
    w = torch.randint(0, 17, (1, 16), generator=b.gen, dtype=torch.int32).cuda()
    kps = torch.tensor([16], dtype=torch.int32).cuda()
    calls = [lambda s: dsa.sparse_attn_decode_fp8(c8, b.seqs, b.queries, q, sel, cnt, stream=s),
             lambda s: dsa.sparse_attn_decode(c16, b.seqs, b.queries, q, sel, cnt, stream=s),
             lambda s: dsa.select_blocks(c16, b.seqs, b.queries, q_idx, w, kps, 16, stream=s),
             lambda s: dsa.topk_blocks(b.seqs, b.queries, dsa.index_score(c16, b.seqs, b.queries, q_idx, w, stream=s), kps,
                                       16, stream=s)]
    side = torch.cuda.Stream()
    for i, call in enumerate(calls):
        want = [t.clone() for t in call(None)]
        _dirty()
        torch.cuda._sleep(BUSY)
        got = call(side)
        side.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y), i
        torch.cuda.synchronize()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_append_reads_rows_that_the_kernel_ahead_writes(fp8, cuda_device):
    """The appended rows and queries are the output of a long kernel just before that lets its
    successors start early (an attention call), directly and with a short library call between."""
    T = 600
    b = Batch((900, 900), (300, 300), 8, 64, seed=102)
    _, src = b.cache8()
    sel, cnt = (t.cuda() for t in selection(b, 12))
    _, cache = b.cache8() if fp8 else b.cache16()
    _, _, rope = rotary()
    small = Batch((70,), (1,), 1, 1, seed=103)
    _, other = small.cache16()
    # attention output [T][64][128]: heads 0..47 serve as queries, 48..55 as K, 56..63 as V
    out, lse = torch.empty((T, 64, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((T, 64), device="cuda")
    q, k, v = out.split([48, 8, 8], dim=1)
    q_out = torch.empty((T, 48, 128), dtype=torch.bfloat16, device="cuda")
    state = [cache.k_pool, cache.v_pool] + ([cache.k_scale, cache.v_scale] if fp8 else [])
    start = [t.clone() for t in state]

    def attention():
        dsa.sparse_attn_prefill_fp8(src, b.seqs, b.queries, b.dq, sel, cnt, out=out, lse=lse, dev_err=b.err)

    def between():
        dsa.kv_append_rope(other, small.seqs, small.queries.cu_q, small.dk, small.dv, None, rope, dev_err=b.err)

    def append():
        (dsa.kv_append_fp8 if fp8 else dsa.kv_append_rope)(
            cache, b.seqs, b.queries.cu_q, k, v, None, rope, queries=b.queries, q=q, q_out=q_out, dev_err=b.err)

    def restore():
        out.zero_()
        q_out.zero_()
        for t, old in zip(state, start):
            t.copy_(old)
        torch.cuda.synchronize()

    restore()
    attention()
    torch.cuda.synchronize()
    append()
    torch.cuda.synchronize()
    want = [t.clone() for t in [q_out] + state]
    assert bool(want[0].any()) and int(b.err) == 0
    for chain in ((attention, append), (attention, between, append)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for call in chain:
                call()
        for i in range(10):
            restore()
            if i % 2:
                graph.replay()
            else:
                for call in chain:
                    call()
            torch.cuda.synchronize()
            for got, w in zip([q_out] + state, want):
                assert torch.equal(got.view(torch.uint8), w.view(torch.uint8)), i
    assert int(b.err) == 0


def test_a_stream_is_whatever_holds_its_handle(cuda_device):
    """A call's stream may be any object with the handle in cuda_stream, also where the call allocates."""
    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    b, cache, args = _step_case(True, seed=104)
    want = {k: v.clone() for k, v in dsa.step(cache, b.seqs, b.queries, **args).items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for got in (dsa.step(cache, b.seqs, b.queries, stream=Handle(side), **args),
                dsa.PreparedStep(cache, b.seqs, b.queries, stream=Handle(side), **args)()):
        side.synchronize()
        for n in ("sel", "cnt", "out", "lse", "q_rot"):
            assert torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)), n
