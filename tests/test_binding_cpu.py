"""The binding without a device: where a call's allocations are made."""
import contextlib
import ctypes

import torch

import dynamic_block_sparse_dsa_b200 as dsa
from dynamic_block_sparse_dsa_b200 import workloads as wk


class FakeLib:
    """Stands in for the library: sizes are small, every call succeeds."""

    def __getattr__(self, name):
        return (lambda *a: 256) if name.endswith("_workspace_size") else (lambda *a: 0)


class FakeStream:
    cuda_stream = 7


def test_allocations_are_made_on_the_calls_stream(monkeypatch):
    """Every buffer that a call on a given stream allocates is allocated under that stream: a
    workspace whose zero fill ran on another one would race with the call's kernels."""
    inside, made = [], []

    @contextlib.contextmanager
    def on(stream):
        inside.append(stream)
        yield
        inside.pop()

    for name in ("zeros", "empty", "empty_like"):
        real = getattr(torch, name)

        def alloc(*a, _real=real, _name=name, **k):
            made.append((_name, inside[-1] if inside else None))
            return _real(*a, **k)
        monkeypatch.setattr(torch, name, alloc)
    fake, stream = FakeLib(), FakeStream()
    monkeypatch.setattr(dsa._lib, "load", lambda: fake)
    monkeypatch.setattr(dsa, "load", lambda: fake)
    monkeypatch.setattr(dsa, "_on", on)
    monkeypatch.setattr(dsa, "_ptr", lambda t: None if t is None else ctypes.c_void_p(t.data_ptr()))
    monkeypatch.setattr(dsa, "_current", lambda t: -1)
    spec = wk.WorkloadSpec("as", seq_lens=(900, 300), n_new=(1, 1), k_per_seq=(4, 4), k_max=4, num_q_heads=8,
                           num_kv_heads=1, num_idx_heads=4)
    wl = wk.make_workload(spec, seed=3)
    cache = dsa.PagedKVCache(wl.k_pool, wl.v_pool, wl.kc_pool)
    code = torch.zeros(wl.k_pool.shape, dtype=torch.uint8)
    scale = torch.ones(code.shape[0], code.shape[1] // 64, 1)
    cache8 = dsa.PagedKVCacheFP8(code, code, wl.kc_pool, scale, scale)
    seqs, queries = dsa.SeqBatch(wl.block_table, wl.seq_lens), dsa.QueryBatch(wl.cu_q, wl.q_pos)
    kw = dict(k_new=wl.k_new, v_new=wl.v_new, kc_new=wl.kc_new, q=wl.q, q_idx=wl.q_idx, w=wl.w, k_per_seq=wl.k_per_seq,
              k_max=4, stream=stream)
    rope = dsa.Rotary(torch.ones(64))

    def check():
        assert made and all(s is stream for _, s in made), made
        made.clear()

    made.clear()
    for c in (cache, cache8):
        for extra in (dict(), dict(fused_select=True), dict(decode=False), dict(rope=rope)):
            dsa.step(c, seqs, queries, **kw, **extra)
            check()
    for extra in (dict(fused_select=True, overlap_append=True), dict(fused_decode=True)):
        dsa.step(cache, seqs, queries, **kw, **extra)
        check()
    sel, cnt = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    scores = torch.zeros(2, wl.block_table.shape[1], dtype=torch.int32)
    made.clear()
    for call, args in ((dsa.index_score, (cache, seqs, queries, wl.q_idx, wl.w)),
                       (dsa.index_score_i64, (cache, seqs, queries, wl.q_idx, wl.w)),
                       (dsa.index_score_fp8, (cache, seqs, queries, wl.q_idx.view(torch.uint8), wl.w)),
                       (dsa.topk_blocks, (seqs, queries, scores, wl.k_per_seq, 4)),
                       (dsa.topk_blocks_i64, (seqs, queries, scores.long(), wl.k_per_seq, 4)),
                       (dsa.select_blocks, (cache, seqs, queries, wl.q_idx, wl.w, wl.k_per_seq, 4)),
                       (dsa.select_blocks_append, (cache, seqs, queries, wl.cu_q, wl.k_new, wl.v_new, None, wl.q_idx, wl.w,
                                                   wl.k_per_seq, 4)),
                       (dsa.sparse_attn_decode, (cache, seqs, queries, wl.q, sel, cnt)),
                       (dsa.sparse_attn_prefill, (cache, seqs, queries, wl.q, sel, cnt)),
                       (dsa.sparse_attn_decode_noalloc, (cache, seqs, queries, wl.q, sel, cnt)),
                       (dsa.sparse_attn_decode_fp8, (cache8, seqs, queries, wl.q, sel, cnt)),
                       (dsa.sparse_attn_prefill_fp8, (cache8, seqs, queries, wl.q, sel, cnt)),
                       (dsa.decode_fused, (cache, seqs, queries, wl.cu_q, wl.k_new, wl.v_new, None, wl.q_idx, wl.w,
                                           wl.k_per_seq, 4, wl.q))):
        call(*args, stream=stream)
        check()
