"""The binding without a device: where a call's allocations are made, what the
native reader takes, when it is built."""
import contextlib
import ctypes
import sysconfig

import pytest
import torch

import dynamic_block_sparse_dsa_b200 as dsa
from dynamic_block_sparse_dsa_b200 import build
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


def test_the_native_reader_takes_the_form_of_the_entry_point(monkeypatch):
    """A PagedKVCacheFP8 without scales over bf16 pools is refused before any call: the 8-bit entry
    point would read past the bf16 cache's description."""
    if dsa._native is None:
        pytest.skip("the native reader is not built here")
    calls = []
    entry = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * 8)(lambda *a: calls.append(a) or 0)
    at = ctypes.cast(entry, ctypes.c_void_p).value
    dsa.load()
    for name in ("dsa_kv_append_rope", "dsa_kv_append_fp8"):
        monkeypatch.setitem(dsa._lib.ADDRESS, name, at)
    monkeypatch.setattr(dsa, "_current", lambda t: -1)
    monkeypatch.setattr(dsa, "_raw_stream", lambda s, dev: 0)
    pool = torch.zeros(2, 64, 1, 128, dtype=torch.bfloat16)
    code, kc, scale = torch.zeros(2, 64, 1, 128, dtype=torch.uint8), torch.zeros(2, 64, dtype=torch.int8), torch.ones(2, 1, 1)
    seqs = dsa.SeqBatch(torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    cu, row = torch.tensor([0, 1], dtype=torch.int32), torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    for bad in (dsa.PagedKVCacheFP8(pool, pool, kc, None, None), dsa.PagedKVCacheFP8(pool, pool, kc, scale, scale),
                dsa.PagedKVCacheFP8(code, code, kc, None, None), dsa.PagedKVCacheFP8(code, code, kc, scale, None)):
        with pytest.raises((ValueError, AttributeError)):
            dsa.kv_append_fp8(bad, seqs, cu, row, row)
    with pytest.raises(ValueError):
        dsa.kv_append_rope(dsa.PagedKVCache(code, code, kc), seqs, cu, row, row, None, dsa.Rotary(torch.ones(64)))
    assert not calls
    dsa.kv_append_fp8(dsa.PagedKVCacheFP8(code, code, kc, scale, scale), seqs, cu, row, row)
    dsa.kv_append_rope(dsa.PagedKVCache(pool, pool, kc), seqs, cu, row, row, None, dsa.Rotary(torch.ones(64)))
    assert len(calls) == 2


# ----------------------------------------------------------------------------- the native reader's build

def test_the_reader_is_stale_when_anything_it_is_built_from_changes(monkeypatch, tmp_path):
    """Its source, the header whose structs it fills, torch: each makes a built reader stale; and its
    file is named for this Python."""
    if not build.build_tensor_args():
        pytest.skip("no C++ compiler here")
    assert not build.args_stale()
    assert build.ARGS_LIB.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    for name in ("HEADER", "ARGS_SRC"):
        with monkeypatch.context() as m:
            other = tmp_path / name
            other.write_text(open(getattr(build, name)).read() + "\n/* another field */\n")
            m.setattr(build, name, str(other))
            assert build.args_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        assert build.args_stale()
    assert not build.args_stale()


def test_a_stale_reader_is_not_used_and_one_built_here_is(monkeypatch):
    from dynamic_block_sparse_dsa_b200 import _args
    if _args.native is None and not build.build_tensor_args():
        pytest.skip("no C++ compiler here")
    for m, names in ((_args, ("native", "_at", "_rows")), (dsa, ("_native", "_at", "_rows"))):
        for n in names:
            monkeypatch.setattr(m, n, None)
    monkeypatch.setattr(build, "args_stale", lambda: True)
    monkeypatch.setattr(build, "build_tensor_args", lambda: False)
    _args.connect()
    dsa._connect()
    assert _args.native is None and dsa._native is None      # stale, and not to be built
    monkeypatch.setattr(build, "build_tensor_args", lambda: True)
    _args.connect()
    assert _args.native is None                              # an import builds nothing
    dsa._connect()                                           # as load() does
    assert _args.native is not None and dsa._native is _args.native and dsa._at is _args.native.at
    monkeypatch.setattr(_args, "native", None)
    monkeypatch.setattr(build, "args_key", lambda: "another")
    _args.connect(build=True)
    assert _args.native is None                              # the module in this process is not the one just built


def test_selection_over_the_8bit_cache_checks_the_coarse_keys():
    """The indexer and selection calls read one 64-byte row per page: a kc_pool of wider elements or
    of fewer rows would be read as something else, or past its end."""
    code, scale = torch.zeros(2, 64, 1, 128, dtype=torch.uint8), torch.ones(2, 1, 1)
    seqs = dsa.SeqBatch(torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    queries = dsa.QueryBatch(torch.tensor([0, 1], dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    q_idx, w = torch.zeros(1, 4, 64, dtype=torch.int8), torch.zeros(1, 4, dtype=torch.int32)
    kps = torch.ones(1, dtype=torch.int32)
    for kc in (torch.zeros(1, 64, dtype=torch.int8), torch.zeros(2, 64, dtype=torch.int32)):
        cache = dsa.PagedKVCacheFP8(code, code, kc, scale, scale)
        for call in (lambda: dsa.index_score(cache, seqs, queries, q_idx, w),
                     lambda: dsa.select_blocks(cache, seqs, queries, q_idx, w, kps, 1, workspace=torch.zeros(1))):
            with pytest.raises(ValueError, match="one row per page"):
                call()
