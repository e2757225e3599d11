"""Host checks of the rotary append and the 8-bit cache (no device needed):
the C entry points refuse bad arguments before any CUDA call, and the binding
refuses what it cannot pass on."""
import ctypes

import pytest
import torch

import dynamic_block_sparse_dsa_b200 as dsa
from dynamic_block_sparse_dsa_b200 import _lib

FAKE = 0x10000   # a 16-byte aligned address that is never dereferenced on these paths
BAD, UNSUP = _lib.DSA_ERR_INVALID_ARG, _lib.DSA_ERR_UNSUPPORTED


def _make(cls, base, kw):
    base = dict(base)
    base.update(kw)
    return cls(**base)


def cache(**kw):
    return _make(_lib.KvCacheC, dict(k_pool=FAKE, v_pool=FAKE, kc_pool=FAKE, num_pages=4, block_size=64,
                                     num_kv_heads=8, head_dim=128, idx_dim=64), kw)


def cache8(**kw):
    return _make(_lib.KvCacheFp8C, dict(k_pool=FAKE, v_pool=FAKE, kc_pool=FAKE, k_scale=FAKE, v_scale=FAKE,
                                        num_pages=4, block_size=64, num_kv_heads=8, head_dim=128, idx_dim=64), kw)


def seqs(**kw):
    return _make(_lib.SeqsC, dict(block_table=FAKE, max_blocks=4, seq_lens=FAKE, num_seqs=1), kw)


def queries(**kw):
    return _make(_lib.QueriesC, dict(cu_q=FAKE, q_pos=FAKE, total_q=1), kw)


def fresh(**kw):
    return _make(_lib.NewTokensC, dict(cu_new=FAKE, total_new=1, k=FAKE, v=FAKE, k_stride=1024, v_stride=1024,
                                       kc=None, pos=None), kw)


def rope(**kw):
    return _make(_lib.RopeC, dict(inv_freq=FAKE, pair_axis=None, rotary_dim=128, layout=0, num_axes=1, scale=1.0), kw)


def rows(**kw):
    return _make(_lib.QueryRowsC, dict(q=FAKE, q_stride=8192, num_heads=64, pos=None, out=FAKE + 65536), kw)


def ref(x):
    return None if x is None else ctypes.byref(x)


def append(fn, c, s=None, f=None, r=rope(), q=None, w=None):
    return getattr(_lib.load(), fn)(ref(c), ref(s or seqs()), ref(f or fresh()), ref(r), ref(q), ref(w), None, None)


ENTRIES = [("dsa_kv_append_rope", cache), ("dsa_kv_append_fp8", cache8)]


@pytest.mark.parametrize("fn,mk", ENTRIES)
def test_append_refusals(fn, mk):
    assert append(fn, mk(block_size=96)) == UNSUP
    assert append(fn, mk(head_dim=64)) == UNSUP
    assert append(fn, mk(k_pool=FAKE + 8)) == BAD
    assert append(fn, mk(num_pages=0)) == BAD
    assert append(fn, mk(), s=seqs(block_table=None)) == BAD
    assert append(fn, mk(), f=fresh(total_new=-1)) == BAD
    assert append(fn, mk(), f=fresh(k=None)) == BAD
    assert append(fn, mk(), f=fresh(v=FAKE + 2)) == BAD
    assert append(fn, mk(), f=fresh(kc=FAKE + 8)) == BAD
    assert append(fn, mk(), f=fresh(k_stride=1016)) == BAD        # less than a token's rows
    assert append(fn, mk(), f=fresh(v_stride=1028)) == BAD        # rows would lose their alignment
    for bad in (dict(rotary_dim=0), dict(rotary_dim=130), dict(inv_freq=None), dict(layout=2), dict(num_axes=0),
                dict(num_axes=2), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert append(fn, mk(), r=rope(**bad)) == BAD, bad
    assert append(fn, mk(), r=rope(rotary_dim=24)) == UNSUP
    assert append(fn, mk(), r=rope(num_axes=5, pair_axis=FAKE)) == UNSUP
    for bad in (dict(q=None), dict(out=None), dict(num_heads=0), dict(q=FAKE + 2), dict(out=FAKE + 8),
                dict(q_stride=8184), dict(q_stride=8196), dict(out=FAKE, q_stride=16384)):
        assert append(fn, mk(), q=queries(), w=rows(**bad)) == BAD, bad
    assert append(fn, mk(), q=queries(total_q=-1), w=rows()) == BAD
    assert append(fn, mk(), q=None, w=rows()) == BAD
    # nothing to do is fine and launches nothing
    assert append(fn, mk(), f=fresh(total_new=0)) == _lib.DSA_OK
    assert append(fn, mk(), f=fresh(total_new=0), q=queries(total_q=0), w=rows(q=None)) == _lib.DSA_OK


def test_rotation_is_optional_for_the_8bit_append_only():
    assert append("dsa_kv_append_rope", cache(), f=fresh(total_new=0), r=None) == BAD
    assert append("dsa_kv_append_fp8", cache8(), f=fresh(total_new=0), r=None) == _lib.DSA_OK
    assert append("dsa_kv_append_fp8", cache8(), r=None, q=queries(), w=rows()) == BAD   # queries unchanged
    assert append("dsa_kv_append_fp8", cache8(k_scale=None)) == BAD
    assert append("dsa_kv_append_fp8", cache8(v_scale=FAKE + 4)) == BAD


def test_fp8_attention_refusals():
    lib = _lib.load()
    s, q = seqs(), queries()

    def dec(c=None, hq=64, k_max=32, ws=FAKE, ws_bytes=1 << 30, scale=0.088, qq=q):
        return lib.dsa_sparse_attn_decode_fp8(ref(c or cache8()), ref(s), ref(qq), FAKE, hq, FAKE, FAKE, k_max, scale,
                                              FAKE, None, ws, ws_bytes, None, None)

    def pre(c=None, hq=64, k_max=32, scale=0.088, qq=q):
        return lib.dsa_sparse_attn_prefill_fp8(ref(c or cache8()), ref(s), ref(qq), FAKE, hq, FAKE, FAKE, k_max,
                                               scale, FAKE, None, None, None)

    for call in (dec, pre):
        assert call(cache8(k_scale=None)) == BAD
        assert call(cache8(v_scale=None)) == BAD
        assert call(cache8(block_size=32)) == UNSUP
        assert call(hq=60) == BAD                # not a multiple of the KV heads
        assert call(hq=8 * 17) == UNSUP          # group of 17
        assert call(k_max=0) == BAD
        assert call(scale=0.0) == BAD
        assert call(scale=float("nan")) == BAD
        assert call(cache8(num_pages=1 << 25)) == UNSUP          # pool rows past 31 bits
        assert call(qq=queries(total_q=1 << 22), k_max=64) == UNSUP   # work units past 31 bits
        assert call(qq=queries(total_q=0)) == _lib.DSA_OK
    assert dec(ws=None) == _lib.DSA_ERR_WORKSPACE
    assert dec(ws=FAKE + 8) == _lib.DSA_ERR_WORKSPACE
    assert dec(ws_bytes=1024) == _lib.DSA_ERR_WORKSPACE


# ----------------------------------------------------------------------------- the binding

def _host():
    c8 = dsa.PagedKVCacheFP8(torch.zeros(2, 64, 1, 128, dtype=torch.uint8), torch.zeros(2, 64, 1, 128, dtype=torch.uint8),
                             torch.zeros(2, 64, dtype=torch.int8), torch.ones(2, 1, 1), torch.ones(2, 1, 1))
    c16 = dsa.PagedKVCache(torch.zeros(2, 64, 1, 128, dtype=torch.bfloat16),
                           torch.zeros(2, 64, 1, 128, dtype=torch.bfloat16), torch.zeros(2, 64, dtype=torch.int8))
    s = dsa.SeqBatch(torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    q = dsa.QueryBatch(torch.tensor([0, 1], dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    row = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    return c8, c16, s, q, row


def test_binding_refuses_host_tensors_and_the_wrong_cache():
    c8, c16, s, q, row = _host()
    r = dsa.Rotary(torch.ones(64))
    sel, cnt = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        dsa.kv_append_fp8(c8, s, q.cu_q, row, row, None, r)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        dsa.kv_append_rope(c16, s, q.cu_q, row, row, None, r)
    for call in (dsa.sparse_attn_decode_fp8, dsa.sparse_attn_prefill_fp8):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call(c8, s, q, row, sel, cnt)
        with pytest.raises(TypeError):
            call(c16, s, q, row, sel, cnt)
    with pytest.raises(TypeError):
        dsa.kv_append_rope(c8, s, q.cu_q, row, row, None, r)
    with pytest.raises(TypeError):
        dsa.kv_append_fp8(c16, s, q.cu_q, row, row)
    # a bf16 append would write two bytes per code: the 8-bit cache is not taken for a bf16 one
    with pytest.raises(TypeError, match="bf16 PagedKVCache"):
        dsa.kv_append(c8, s, q.cu_q, row, row)
    with pytest.raises(TypeError, match="bf16 PagedKVCache"):
        dsa.sparse_attn_prefill(c8, s, q, row, sel, cnt)
    for kw in (dict(overlap_append=True, fused_select=True), dict(fused_decode=True)):
        with pytest.raises(ValueError, match="rotated already"):
            dsa.step(c8, s, q, k_new=row, v_new=row, kc_new=None, q=row, q_idx=None, w=None, k_per_seq=None, k_max=1,
                     **kw)
    with pytest.raises(ValueError, match="pos needs rope"):
        dsa.step(c8, s, q, k_new=row, v_new=row, kc_new=None, q=row, q_idx=None, w=None, k_per_seq=None, k_max=1,
                 pos=q.q_pos)


def test_binding_refuses_mismatched_shapes():
    c8, c16, s, q, row = _host()
    for bad in (dict(k_scale=torch.ones(2, 1, 2)), dict(v_scale=torch.ones(2, 2, 1)),
                dict(k_scale=torch.ones(2, 1, 1, dtype=torch.float64)),
                dict(k_pool=torch.zeros(2, 64, 1, 128, dtype=torch.bfloat16)),
                dict(v_pool=torch.zeros(2, 64, 2, 128, dtype=torch.uint8)),
                dict(kc_pool=torch.zeros(1, 64, dtype=torch.int8))):
        kw = dict(k_pool=c8.k_pool, v_pool=c8.v_pool, kc_pool=c8.kc_pool, k_scale=c8.k_scale, v_scale=c8.v_scale)
        kw.update(bad)
        with pytest.raises(ValueError):
            dsa.PagedKVCacheFP8(**kw).packed(-1)
    with pytest.raises(ValueError, match="pair_axis"):
        dsa.Rotary(torch.ones(64), num_axes=3).packed(-1)
    with pytest.raises(ValueError, match="pair_axis"):
        dsa.Rotary(torch.ones(64), num_axes=2, pair_axis=torch.zeros(32, dtype=torch.int32)).packed(-1)
    with pytest.raises(ValueError, match="float32"):
        dsa.Rotary(torch.ones(64, dtype=torch.float64)).packed(-1)
    with pytest.raises(ValueError, match="seq_lens"):
        dsa.SeqBatch(s.block_table, torch.ones(2, dtype=torch.int32)).packed(-1)
    with pytest.raises(ValueError, match="contiguous"):
        dsa.SeqBatch(torch.zeros(2, 4, dtype=torch.int32)[:, ::2], torch.ones(2, dtype=torch.int32)).packed(-1)
    with pytest.raises(ValueError, match="other tensors"):
        dsa._at(row, torch.bfloat16, 0, "row") if row.get_device() >= 0 else dsa._wrong_device(1, 0, "row")


def test_native_tensor_reader_answers_as_the_python_one():
    """Same addresses and strides, same refusals, for contiguous and sliced, empty and
    single-token, wrongly typed and wrongly shaped tensors (on the CPU: device -1)."""
    from dynamic_block_sparse_dsa_b200 import _args
    from dynamic_block_sparse_dsa_b200 import build as b
    if not b.build_tensor_args():
        pytest.skip("no C++ compiler here")
    native = pytest.importorskip("dynamic_block_sparse_dsa_b200._tensor_args")
    native.use(_args.py_at, _args.py_rows)

    def both(f, g, *a):
        got = []
        for h in (f, g):
            try:
                got.append(h(*a))
            except Exception as e:
                got.append((type(e), str(e)))
        assert got[0] == got[1], (a, got)
        return got[0]

    x = torch.zeros(5, 6, 128, dtype=torch.bfloat16)
    for t in (x, x[:, 1:3], x[:1], x[:1, 2:3], x[:, :, :64], x.transpose(0, 1), x[::2], x[:0], x.float(), x[0], x[..., ::2]):
        both(native.rows, _args.py_rows, t, -1, "x")
        both(native.at, _args.py_at, t, torch.bfloat16, -1, "x")
        both(native.at, _args.py_at, t, torch.bfloat16, 0, "x")
        both(native.rows, _args.py_rows, t, 0, "x")
    assert both(native.rows, _args.py_rows, x[:, 1:3], -1, "x") == (x.data_ptr() + 256, 5, 2, 768)
    assert both(native.at, _args.py_at, None, torch.int32, -1, "x")[0] is AttributeError


def test_packed_structs_have_the_c_layout():
    """The packed bytes are the ctypes structures' bytes (up to the padding at their end)."""
    def same(packed, c):
        raw = bytes(c)
        assert raw[:len(packed)] == packed and len(raw) - len(packed) < 8

    same(_lib.pack_cache(1, 2, 3, 4, 5, 6, 7, 8), _lib.KvCacheC(1, 2, 3, 4, 5, 6, 7, 8))
    same(_lib.pack_cache_fp8(1, 2, 3, 4, 5, 6, 7, 8, 9, 10), _lib.KvCacheFp8C(1, 2, 3, 4, 5, 6, 7, 8, 9, 10))
    same(_lib.pack_seqs(1, 2, 3, 4), _lib.SeqsC(1, 2, 3, 4))
    same(_lib.pack_queries(1, 2, 3), _lib.QueriesC(1, 2, 3))
    same(_lib.pack_rope(1, 2, 3, 4, 5, 0.5), _lib.RopeC(1, 2, 3, 4, 5, 0.5))
    same(_lib.pack_new_tokens(1, 2, 3, 4, 5, 6, 7, 8), _lib.NewTokensC(1, 2, 3, 4, 5, 6, 7, 8))
    same(_lib.pack_query_rows(1, 2, 3, 4, 5), _lib.QueryRowsC(1, 2, 3, 4, 5))
