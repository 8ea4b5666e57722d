"""Refusals of the layer-step operators, on the host: bad arguments are turned
down before anything is launched."""
import ctypes

import pytest
import torch

import paged_kv_cache_452_b200 as pa

P = 4096  # an aligned address that is never read: every call here returns first


def write(desc, prep, n=1, q=P, qs=1 << 14, k=2 * P, ks=1 << 14, v=3 * P, vs=1 << 14, pos=P, slots=P, out=1 << 30, kc=P,
          vc=P):
    return pa.lib().pa_norm_rope_write(ctypes.byref(desc) if desc is not None else None,
                                       ctypes.byref(prep) if prep is not None else None, q, qs, k, ks, v, vs, pos, slots,
                                       n, out, kc, vc, None)


def prep_of(qw=P, kw=P, eps=1e-6, cs=P, npos=10, rot=64, inter=0):
    return pa.QkPrep(qw, kw, eps, cs, npos, rot, inter)


def test_norm_rope_write_refusals():
    desc = pa.CacheDesc.make(16, 16, 2, 8, 64, "bf16", "bf16")
    assert write(None, prep_of()) == 1
    assert write(desc, None) == 1
    assert write(desc, prep_of(), n=0) == 0 and write(desc, prep_of(), n=-1) == 1
    for bad in (prep_of(eps=-1.0), prep_of(eps=float("nan")), prep_of(npos=0), prep_of(rot=0), prep_of(rot=12),
                prep_of(rot=72), prep_of(inter=2), prep_of(qw=P + 8), prep_of(kw=P + 2), prep_of(cs=P + 4)):
        assert write(desc, bad) == 1
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(pos=None), dict(slots=None), dict(out=None), dict(kc=None),
               dict(vc=None), dict(q=P + 8), dict(k=P + 2), dict(pos=P + 2), dict(slots=P + 4), dict(out=P + 4),
               dict(qs=8 * 64 - 8), dict(ks=2 * 64 - 8), dict(vs=129), dict(qs=(1 << 28) + 8)):
        assert write(desc, prep_of(), n=3, **kw) == 1, kw
    # q_out over an input: in place only when q's rows lie end to end
    assert write(desc, prep_of(), n=3, out=P) == 1
    assert b"overlaps" in pa.lib().pa_last_error()
    assert write(desc, prep_of(), n=3, out=2 * P + 16) == 1
    assert write(pa.CacheDesc.make(16, 16, 2, 8, 64, "f32", "bf16"), prep_of()) == 2
    assert write(pa.CacheDesc.make(16, 16, 2, 8, 96, "bf16", "bf16"), prep_of()) == 2


def test_cache_read_refusals():
    desc = pa.CacheDesc.make(16, 16, 2, 8, 64, "bf16", "bf16")

    def read(d, n=1, slots=P, kc=P, vc=P, ko=P, vo=P):
        return pa.lib().pa_cache_read(ctypes.byref(d) if d is not None else None, slots, n, kc, vc, ko, vo, None)
    assert read(None) == 1 and read(desc, n=-1) == 1 and read(desc, n=0) == 0
    for kw in (dict(slots=None), dict(kc=None), dict(vc=None), dict(ko=None), dict(vo=None), dict(slots=P + 4),
               dict(ko=P + 8), dict(vc=P + 2)):
        assert read(desc, **kw) == 1, kw
    assert read(pa.CacheDesc.make(16, 16, 2, 8, 64, "bf16", "f32")) == 2


def test_bindings_refuse_wrong_tensors():
    desc = pa.CacheDesc.make(4, 16, 2, 8, 64, "bf16", "bf16")
    bf = torch.bfloat16
    kc, vc = pa.alloc_cache(desc, "cpu")
    q, k, v, out = (torch.zeros((3, h, 64), dtype=bf) for h in (8, 2, 2, 8))
    slots, pos = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    cs, w = torch.zeros((10, 64)), torch.zeros(64, dtype=bf)
    prep = pa.QkPrep.make(w, w, 1e-6, cs)
    good = dict(q=q, k=k, v=v, positions=pos, slot_mapping=slots, q_out=out, k_cache=kc, v_cache=vc)
    with pytest.raises(pa.PaError, match="CUDA device"):  # all well but for the place
        pa.pa_norm_rope_write(desc, prep, **good)
    for bad in (dict(q=q.float()), dict(k=k[:2]), dict(v=v[:, :1]), dict(q=q.transpose(1, 2)), dict(slot_mapping=pos),
                dict(positions=slots), dict(positions=None), dict(q_out=out[:, :, ::2]), dict(k_cache=kc[:3]),
                dict(v_cache=vc.float()), dict(q_out=torch.zeros((3, 16, 64), dtype=bf)[:, ::2])):
        with pytest.raises(pa.PaError, match="pa_norm_rope_write"):
            pa.pa_norm_rope_write(desc, prep, **{**good, **bad})
        assert "CUDA device" not in str(pytest.raises(pa.PaError, pa.pa_norm_rope_write, desc, prep,
                                                      **{**good, **bad}).value)
    with pytest.raises(pa.PaError, match="q_weight"):
        pa.pa_norm_rope_write(desc, pa.QkPrep.make(w.float(), w.float(), 1e-6, cs), **good)
    with pytest.raises(pa.PaError, match="cos_sin"):
        pa.QkPrep.make(w, w, 1e-6, cs.double())
    with pytest.raises(pa.PaError, match="weights"):
        pa.QkPrep.make(w, w.float(), 1e-6, cs)
    with pytest.raises(pa.PaError, match="k_out"):
        pa.pa_cache_read(desc, slots, kc, vc, k[:2], v)
    with pytest.raises(pa.PaError, match="CUDA device"):
        pa.pa_cache_read(desc, slots, kc, vc, k, v)


def test_biased_attention_refusals():
    desc = pa.CacheDesc.make(16, 16, 2, 8, 64, "bf16", "bf16")
    f32 = pa.CacheDesc.make(16, 16, 2, 8, 64, "f32", "f32")
    L = pa.lib()
    mod = pa.ScoreMod(30.0, 10, P, P)

    def decode(d, m, q=P, kc=P, vc=P, bt=P, mb=4, sl=P, n=2, scale=0.125, out=P, ws=P, wb=1 << 30):
        return L.pa_decode_biased(ctypes.byref(d) if d is not None else None, ctypes.byref(m) if m is not None else None,
                                  q, kc, vc, bt, mb, sl, n, scale, out, ws, wb, None)

    def chunk(d, m, q=P, kc=P, vc=P, bt=P, mb=4, qsl=P, sl=P, n=2, t=5, mq=4, scale=0.125, out=P, ws=P, wb=1 << 30):
        return L.pa_decode_chunked_prefill_biased(
            ctypes.byref(d) if d is not None else None, ctypes.byref(m) if m is not None else None, q, kc, vc, bt, mb,
            qsl, sl, n, t, mq, scale, out, ws, wb, None)
    bad_mods = [pa.ScoreMod(-1.0, 0, None, None), pa.ScoreMod(float("nan"), 0, None, None),
                pa.ScoreMod(float("inf"), 0, None, None), pa.ScoreMod(2e4, 0, None, None),
                pa.ScoreMod(1e-5, 0, None, None), pa.ScoreMod(0.0, -1, None, None),
                pa.ScoreMod(0.0, 0, P + 2, None), pa.ScoreMod(0.0, 0, None, P + 1)]
    for call in (decode, chunk):
        assert call(None, mod) == 1 and call(desc, None) == 1
        for m in bad_mods:
            assert call(desc, m) == 1
        for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(bt=None), dict(sl=None), dict(out=None), dict(ws=None),
                   dict(q=P + 8), dict(out=P + 2), dict(ws=P + 16), dict(n=-1), dict(mb=-1), dict(scale=0.0),
                   dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
            assert call(desc, mod, **kw) == 1, kw
        assert call(desc, mod, scale=1e21) == 1  # with a cap
        assert call(f32, mod, wb=255) == 1  # workspace too small, fp32 path
        assert call(desc, mod, n=20000) == 2
        assert call(desc, mod, n=1, mb=1 << 27) == 2  # a table row of 2^31 tokens
        assert call(desc, mod, n=0) == 0
    for kw in (dict(qsl=None), dict(qsl=P + 2), dict(t=-1), dict(mq=-1), dict(mq=0)):
        assert chunk(desc, mod, **kw) == 1, kw
    assert chunk(desc, mod, t=0) == 0
    assert L.pa_biased_workspace_size(ctypes.byref(desc), -1, 1) == 0
    assert L.pa_biased_workspace_size(None, 1, 1) == 0
    assert pa.pa_biased_workspace_size(f32, 4, 4) == 256


@pytest.mark.parametrize("kv,q", [("f32", "bf16"), ("bf16", "f32")])
def test_biased_attention_refuses_pairs_that_are_not_built(kv, q):
    """bf16 queries over an fp32 pool, or fp32 queries over a bf16 pool: no kernel reads them, and none is launched."""
    desc = pa.CacheDesc.make(16, 16, 2, 8, 64, kv, q)
    L, d, m = pa.lib(), ctypes.byref(desc), ctypes.byref(pa.ScoreMod(30.0, 10, None, None))
    assert L.pa_decode_biased(d, m, P, P, P, P, 4, P, 2, 0.125, P, P, 1 << 30, None) == 2
    assert b"kv dtype" in L.pa_last_error()
    for max_q_len in (1, 4):
        assert L.pa_decode_chunked_prefill_biased(d, m, P, P, P, P, 4, P, P, 2, 5, max_q_len, 0.125, P, P, 1 << 30,
                                                  None) == 2
    assert L.pa_biased_workspace_size(d, 2, 5) == 0
    with pytest.raises(pa.PaError, match="kv dtype"):
        pa.pa_biased_workspace_size(desc, 2, 5)


def test_biased_steps_check_sizes_before_the_first_launch():
    """Sizes that a later kernel of a step could not take are turned down with the arguments, ahead of the device."""
    mod = ctypes.byref(pa.ScoreMod(30.0, 10, None, None))

    def chunk(desc, n, mb, t, mq):
        return pa.lib().pa_decode_chunked_prefill_biased(ctypes.byref(desc), mod, P, P, P, P, mb, P, P, n, t, mq, 0.125, P,
                                                         P, 1 << 40, None)
    # a group of 16 is two kernel heads per kv head: 2^31 tiles although num_seqs * max_blocks * kv heads is below
    wide = pa.CacheDesc.make(64, 16, 8, 128, 64, "bf16", "bf16")
    assert chunk(wide, 16000, 10000, 20000, 300) == 2 and b"2^31" in pa.lib().pa_last_error()
    assert pa.lib().pa_decode_biased(ctypes.byref(wide), mod, P, P, P, P, 10000, P, 16000, 0.125, P, P, 1 << 40, None) == 2
    # ... which no kernel indexes in a step of full chunks: as far as the device, which this test does not have
    if not torch.cuda.is_available():
        assert chunk(wide, 16000, 10000, 32000, 2) == 4
    # 2^31 units of chunk rows
    many = pa.CacheDesc.make(64, 16, 512, 512, 64, "bf16", "bf16")
    assert chunk(many, 2, 4, 2**30 + 2**21, 2**30) == 2 and b"chunks" in pa.lib().pa_last_error()
    # fp32: the grids of the row kernel and of the tile kernel
    f32 = pa.CacheDesc.make(64, 16, 1, 70000, 64, "f32", "f32")
    assert chunk(f32, 2, 4, 100, 50) == 2
    f32 = pa.CacheDesc.make(64, 16, 1, 1024, 64, "f32", "f32")
    assert chunk(f32, 2, 4, 2**28, 2**27) == 2


def test_a_step_without_rows_needs_no_queries():
    """A step of sequences that all have no new rows: its q and out are empty tensors, whose address is NULL."""
    desc = pa.CacheDesc.make(16, 16, 2, 8, 64, "bf16", "bf16")
    mod = pa.ScoreMod(30.0, 10, None, None)

    def chunk(t, q, out, n=2):
        return pa.lib().pa_decode_chunked_prefill_biased(ctypes.byref(desc), ctypes.byref(mod), q, P, P, P, 4, P, P, n, t, 1,
                                                         0.125, out, P, 1 << 30, None)
    assert chunk(0, None, None) == 0 and chunk(0, None, None, n=0) == 0
    assert chunk(1, None, P) == 1 and chunk(1, P, None) == 1 and chunk(-1, None, None) == 1


def test_a_window_past_32_bits_is_refused():
    for window in (2**31, 2**32 + 5, -1):
        with pytest.raises(pa.PaError, match="window"):
            pa.ScoreMod.make(window=window)
    assert pa.ScoreMod.make(window=2**31 - 1).window == 2**31 - 1


def test_biased_bindings_refuse_wrong_tensors():
    bf, i32 = torch.bfloat16, torch.int32
    desc = pa.CacheDesc.make(4, 16, 2, 8, 64, "bf16", "bf16")
    kc, vc = pa.alloc_cache(desc, "cpu")
    good = dict(q=torch.zeros((2, 8, 64), dtype=bf), k_cache=kc, v_cache=vc, block_tables=torch.zeros((2, 3), dtype=i32),
                seq_lens=torch.zeros(2, dtype=i32), scale=0.125, out=torch.zeros((2, 8, 64), dtype=bf),
                workspace=torch.zeros(1024, dtype=torch.uint8))
    mod = pa.ScoreMod.make(30.0, 0, torch.zeros(8), torch.zeros(2, dtype=i32))
    bad = [dict(q=good["q"].float()), dict(q=good["q"][:1]), dict(out=good["out"][:, :4]), dict(k_cache=kc[:2]),
           dict(block_tables=good["block_tables"].long()), dict(block_tables=good["block_tables"][0]),
           dict(seq_lens=good["seq_lens"].long())]
    bad_mods = [pa.ScoreMod.make(slopes=torch.zeros(4)), pa.ScoreMod.make(prefix_lens=torch.zeros(3, dtype=i32))]
    for kw in (dict(slopes=torch.zeros(8).double()), dict(prefix_lens=torch.zeros(2)), dict(slopes=torch.zeros(16)[::2])):
        with pytest.raises(pa.PaError, match="ScoreMod"):
            pa.ScoreMod.make(**kw)
    chunk = dict(query_start_loc=torch.zeros(3, dtype=i32), max_q_len=1)
    for f, more in ((pa.pa_decode_biased, {}), (pa.pa_decode_chunked_prefill_biased, chunk)):
        with pytest.raises(pa.PaError, match="CUDA device"):
            f(desc, mod, **good, **more)
        for kw in bad:
            assert "CUDA device" not in str(pytest.raises(pa.PaError, f, desc, mod, **{**good, **more, **kw}).value)
        for m in bad_mods:
            assert "CUDA device" not in str(pytest.raises(pa.PaError, f, desc, m, **good, **more).value)
    with pytest.raises(pa.PaError, match="query_start_loc"):
        pa.pa_decode_chunked_prefill_biased(desc, mod, **good, query_start_loc=torch.zeros(2, dtype=i32), max_q_len=1)
