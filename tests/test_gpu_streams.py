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
