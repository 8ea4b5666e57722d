"""pa_norm_rope_write and pa_cache_read against plain fp64 arithmetic on the
same inputs.

Tolerances.  A value y is computed in fp32 from exact inputs: the mean square
and the products keep within a few fp32 roundings of the fp64 value, taken as
2^-19 relative to the row's largest |y| (D = 128 summands, the rsqrt and two
products of a rotation: well under 32 roundings of 2^-24).  The stored value is
off by half a step more: eps/2 relative in bf16 (2^-8) and fp32 (2^-24), and in
e4m3 half a step of the code's grid (2^-4 relative, 2^-10 absolute below the
smallest normal code)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_452_b200 as pa

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0**-24, "bf16": 2.0**-8}
KS, VS = 0.0125, 0.011


def slots_of(n, nb, bs, how, rng):
    if how == "runs":  # whole blocks of consecutive tokens, the first run starting inside a block
        start = int(rng.integers(0, bs))
        need = (n + start + bs - 1) // bs
        flat = (rng.permutation(nb)[:need, None] * bs + np.arange(bs)[None]).reshape(-1)
        return flat[start:start + n].astype(np.int64)
    return rng.permutation(nb * bs)[:n].astype(np.int64)


def fp64_rows(x, w, eps, table, pos, rot, inter):
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    y = y.clone()
    if rot:
        cs = table.double()[pos.long()][:, None]
        cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
        a = (y[..., 0:rot:2] if inter else y[..., :rot // 2]).clone()
        b = (y[..., 1:rot:2] if inter else y[..., rot // 2:rot]).clone()
        if inter:
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def close(got, exp, half, row_slack=2.0**-19):
    """|got - exp| <= half a step of the stored type + the fp32 arithmetic's share."""
    got, exp = got.double(), exp.double()
    top = exp.abs().amax(-1, keepdim=True)
    bad = (got - exp).abs() > half * exp.abs() * (1 + 2.0**-10) + row_slack * top + 1e-30
    assert not bool(bad.any()), float((got - exp).abs().max())


def close_e4m3(codes, exp, scale, head_dim_last=True):
    """codes * 1 against exp / scale on the e4m3 grid."""
    val = codes.view(torch.float8_e4m3fn).double()
    want = (exp.double() / scale).clamp(-448, 448)
    step = torch.maximum(want.abs() * 2.0**-4, torch.full_like(want, 2.0**-10))
    top = want.abs().amax(-1, keepdim=True)
    bad = (val - want).abs() > step * (1 + 2.0**-10) + 2.0**-19 * top
    assert not bool(bad.any()), float((val - want).abs().max())


def setup(n, hq, hkv, d, bs, kv, q, how, dev, seed, strided=True, head_scales=False):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=dev).manual_seed(seed)
    nb = max(4, (n // bs + 2) * 2)
    ksc = vsc = None
    if head_scales:
        ksc = torch.rand(hkv, generator=g, device=dev) * 0.05 + 0.005
        vsc = torch.rand(hkv, generator=g, device=dev) * 0.05 + 0.005
    desc = pa.CacheDesc.make(nb, bs, hkv, hq, d, kv, q, KS, VS, ksc, vsc)
    k_cache, v_cache = pa.alloc_cache(desc, dev)
    for t in (k_cache, v_cache):
        t.view(torch.uint8).random_(0, 100, generator=g)
    qkv = torch.randn((n, hq + 2 * hkv, d), generator=g, device=dev).to(DT[q])
    qkv = qkv * torch.exp(torch.randn((n, hq + 2 * hkv, 1), generator=g, device=dev)).to(DT[q])  # rows of many sizes
    parts = [qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]]
    if not strided:
        parts = [t.contiguous() for t in parts]
    slots = torch.from_numpy(slots_of(n, nb, bs, how, rng)).to(dev)
    return desc, k_cache, v_cache, parts, slots, (ksc, vsc), rng, g


def table_of(positions, rot, dev):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f[None]
    return torch.cat([a.cos(), a.sin()], 1).float().to(dev)


def pool_rows(desc, k_cache, v_cache, slots):
    blk, off = slots // desc.block_size, slots % desc.block_size
    k = k_cache[blk, :, off]
    v = v_cache[blk, :, :, off] if desc.kv_dtype == pa.PA_FP8_E4M3 else v_cache[blk, :, off]
    return k, v


@pytest.mark.parametrize("n,hq,hkv,d,bs,kv,q,rot,inter,how,head_scales", [
    (1, 4, 1, 128, 16, "bf16", "bf16", 128, False, "runs", False),
    (64, 32, 8, 128, 16, "bf16", "bf16", 128, False, "any", False),
    (77, 6, 3, 64, 32, "bf16", "bf16", 16, True, "runs", False),
    (301, 5, 5, 128, 16, "e4m3", "bf16", 64, False, "runs", True),
    (33, 16, 2, 64, 32, "e4m3", "bf16", 64, True, "any", False),
    (45, 3, 1, 64, 16, "e4m3", "f32", 8, False, "runs", False),
    (130, 2, 2, 64, 16, "f32", "f32", 64, False, "runs", False),
    (19, 8, 4, 128, 32, "f32", "f32", 40, True, "any", False),
    (1500, 7, 1, 128, 16, "bf16", "bf16", 0, False, "runs", False),
])
def test_norm_rope_write_matches_fp64(n, hq, hkv, d, bs, kv, q, rot, inter, how, head_scales, cuda_device):
    desc, kc, vc, (xq, xk, xv), slots, (ksc, vsc), rng, g = setup(n, hq, hkv, d, bs, kv, q, how, cuda_device, n,
                                                                  head_scales=head_scales)
    table = table_of(5000, rot, cuda_device) if rot else None
    pos = torch.from_numpy(rng.integers(0, 5000, n).astype(np.int32)).to(cuda_device) if rot else None
    qw = (1 + 0.3 * torch.randn(d, generator=g, device=cuda_device)).to(DT[q])
    kw = (1 + 0.3 * torch.randn(d, generator=g, device=cuda_device)).to(DT[q])
    prep = pa.QkPrep.make(qw, kw, 1e-5, table, inter)
    kb, vb = kc.clone(), vc.clone()
    out = torch.full((n, hq, d), float("nan"), dtype=DT[q], device=cuda_device)
    pa.pa_norm_rope_write(desc, prep, xq, xk, xv, pos, slots, out, kc, vc)
    torch.cuda.synchronize()
    close(out, fp64_rows(xq, qw, 1e-5, table, pos, rot, inter), HALF[q])
    ek = fp64_rows(xk, kw, 1e-5, table, pos, rot, inter)
    gk, gv = pool_rows(desc, kc, vc, slots)
    if kv == "e4m3":
        close_e4m3(gk, ek, KS if ksc is None else ksc.double()[None, :, None])
        close_e4m3(gv, xv.double(), VS if vsc is None else vsc.double()[None, :, None])
        # V as pa_cache_write stores it, to the bit
        k2, v2 = kb.clone(), vb.clone()
        pa.pa_cache_write(desc, xk.contiguous(), xv.contiguous(), slots, k2, v2)
        assert torch.equal(v2, vc)
    else:
        close(gk, ek, HALF[q])
        assert torch.equal(gv, xv)
    # everything else in the pools as it was
    blk, off = slots // bs, slots % bs
    for a, b, dm in ((kb, kc, False), (vb, vc, kv == "e4m3")):
        a, b = a.view(torch.uint8 if kv == "e4m3" else DT[q]), b
        if dm:
            a[blk, :, :, off] = b[blk, :, :, off]
        else:
            a[blk, :, off] = b[blk, :, off]
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def four_row_groups(n, hq, hkv, d):
    """Whether a call has more lanes of work than one launch of the GPU holds: then a row group has four head rows."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return n * (hq + 2 * hkv) * (d // 8) > sms * 2048


@pytest.mark.parametrize("n,hq,hkv,d,bs,kv,q,rot,inter,how,head_scales", [
    (2500, 7, 1, 128, 16, "bf16", "bf16", 128, False, "runs", False),
    (2500, 9, 3, 128, 32, "e4m3", "bf16", 128, False, "runs", True),
    (2500, 9, 1, 128, 16, "e4m3", "f32", 128, False, "runs", False),
    (6000, 6, 3, 64, 16, "f32", "f32", 64, False, "any", False),
    (6000, 5, 5, 64, 32, "e4m3", "bf16", 64, False, "any", False),
    (2500, 6, 3, 128, 16, "e4m3", "bf16", 64, True, "runs", False),
    (6000, 9, 3, 64, 32, "bf16", "bf16", 16, False, "any", False),
    (2500, 10, 2, 128, 16, "f32", "f32", 40, True, "runs", False),
    (2500, 7, 1, 128, 16, "bf16", "bf16", 0, False, "runs", False),
])
def test_norm_rope_write_in_groups_of_four_rows(n, hq, hkv, d, bs, kv, q, rot, inter, how, head_scales, cuda_device):
    """Steps large enough for four head rows per group, head counts that leave a group unfilled, every form of the
    rotation and every pool."""
    assert four_row_groups(n, hq, hkv, d)
    test_norm_rope_write_matches_fp64(n, hq, hkv, d, bs, kv, q, rot, inter, how, head_scales, cuda_device)


@pytest.mark.parametrize("n,hq,hkv,d,bs,q,how,head_scales", [
    (301, 5, 5, 128, 16, "bf16", "runs", True), (77, 6, 3, 64, 32, "bf16", "any", False),
    (45, 3, 1, 64, 16, "f32", "runs", False), (16, 8, 2, 128, 32, "f32", "any", True)])
def test_e4m3_keys_normed_and_rotated_over_the_whole_head(n, hq, hkv, d, bs, q, how, head_scales, cuda_device):
    test_norm_rope_write_matches_fp64(n, hq, hkv, d, bs, "e4m3", q, d, False, how, head_scales, cuda_device)


@pytest.mark.parametrize("n,hq,hkv,d", [(37, 6, 3, 128), (2500, 9, 3, 128), (6000, 6, 3, 64)])
@pytest.mark.parametrize("kv,q", [("bf16", "bf16"), ("e4m3", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("inter,part", [(False, 1), (True, 1), (False, 2)])
def test_rotation_without_a_norm_and_with_one_of_the_two(inter, part, kv, q, n, hq, hkv, d, cuda_device):
    assert four_row_groups(n, hq, hkv, d) == (n > 1000)
    desc, kc, vc, (xq, xk, xv), slots, _, rng, g = setup(n, hq, hkv, d, 16, kv, q, "runs", cuda_device, n + part)
    rot = d // part
    table = table_of(3000, rot, cuda_device)
    pos = torch.from_numpy(rng.integers(0, 3000, n).astype(np.int32)).to(cuda_device)
    kw = (1 + 0.3 * torch.randn(d, generator=g, device=cuda_device)).to(DT[q])
    for w in (None, kw):
        out = torch.full((n, hq, d), float("nan"), dtype=DT[q], device=cuda_device)
        pa.pa_norm_rope_write(desc, pa.QkPrep.make(None, w, 1e-5, table, inter), xq, xk, xv, pos, slots, out, kc, vc)
        close(out, fp64_rows(xq, None, 1e-5, table, pos, rot, inter), HALF[q])
        gk, gv = pool_rows(desc, kc, vc, slots)
        ek = fp64_rows(xk, w, 1e-5, table, pos, rot, inter)
        if kv == "e4m3":
            close_e4m3(gk, ek, KS)
            close_e4m3(gv, xv.double(), VS)
        else:
            close(gk, ek, HALF[q])
            assert torch.equal(gv, xv)


def test_norm_rope_write_without_norm_is_a_rotation_and_a_copy(cuda_device):
    desc, kc, vc, (xq, xk, xv), slots, _, rng, g = setup(37, 8, 2, 128, 16, "bf16", "bf16", "runs", cuda_device, 3)
    out = torch.empty_like(xq, memory_format=torch.contiguous_format)
    pa.pa_norm_rope_write(desc, pa.QkPrep.make(), xq, xk, xv, None, slots, out, kc, vc)
    gk, gv = pool_rows(desc, kc, vc, slots)
    assert torch.equal(out, xq) and torch.equal(gk, xk) and torch.equal(gv, xv)
    # queries alone normed
    w = torch.ones(128, dtype=torch.bfloat16, device=cuda_device)
    pa.pa_norm_rope_write(desc, pa.QkPrep.make(q_weight=w), xq, xk, xv, None, slots, out, kc, vc)
    close(out, fp64_rows(xq, w, 1e-6, None, None, 0, False), HALF["bf16"])
    assert torch.equal(pool_rows(desc, kc, vc, slots)[0], xk)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_norm_rope_write_padding_positions_and_in_place(kv, cuda_device):
    n, hq, hkv, d, bs = 50, 8, 2, 128, 16
    desc, kc, vc, parts, slots, _, rng, g = setup(n, hq, hkv, d, bs, kv, "bf16", "runs", cuda_device, 11, strided=False)
    xq, xk, xv = parts
    table = table_of(100, 128, cuda_device)
    pos = torch.from_numpy(rng.integers(0, 100, n).astype(np.int32)).to(cuda_device)
    w = torch.ones(d, dtype=torch.bfloat16, device=cuda_device)
    prep = pa.QkPrep.make(w, w, 1e-6, table)
    slots[3], slots[17], slots[40] = -1, desc.num_blocks * bs, 2**40  # padding: queries only
    pos[5], pos[41] = -1, 100  # outside the table: left out whole
    want = torch.zeros((n, hq, d), dtype=torch.bfloat16, device=cuda_device)
    full = pos.clone()
    full[5] = full[41] = 0
    k1, v1 = kc.clone(), vc.clone()
    pa.pa_norm_rope_write(desc, prep, xq, xk, xv, full, slots, want, k1, v1)
    keep = xq.clone()
    k0, v0 = kc.clone(), vc.clone()
    pa.pa_norm_rope_write(desc, prep, xq, xk, xv, pos, slots, xq, kc, vc)  # in place
    alive = torch.ones(n, dtype=torch.bool, device=cuda_device)
    alive[5] = alive[41] = False
    assert torch.equal(xq[alive], want[alive]) and torch.equal(xq[~alive], keep[~alive])
    good = alive & (slots >= 0) & (slots < desc.num_blocks * bs)
    for a, b in zip(pool_rows(desc, kc, vc, slots[good]), pool_rows(desc, k1, v1, slots[good])):
        assert torch.equal(a, b)
    for a, b in zip(pool_rows(desc, kc, vc, slots[~alive]), pool_rows(desc, k0, v0, slots[~alive])):
        assert torch.equal(a, b)


def test_norm_rope_write_zero_and_far_rows(cuda_device):
    """A row of zeros stays zero (eps keeps the norm finite); huge and tiny rows norm to the same."""
    desc = pa.CacheDesc.make(8, 16, 1, 1, 128, "bf16", "bf16")
    kc, vc = pa.alloc_cache(desc, cuda_device, fill=0)
    base = torch.randn(128, device=cuda_device).to(torch.bfloat16)
    x = torch.stack([base * 0, base, base * 2.0**30, base * 2.0**-8])[:, None]
    w = torch.ones(128, dtype=torch.bfloat16, device=cuda_device)
    out = torch.empty_like(x)
    slots = torch.arange(4, device=cuda_device)
    pa.pa_norm_rope_write(desc, pa.QkPrep.make(w, w, 1e-6), x, x, x, None, slots, out, kc, vc)
    assert torch.equal(out[0], x[0])
    close(out, fp64_rows(x, w, 1e-6, None, None, 0, False), HALF["bf16"])


@pytest.mark.parametrize("n,hkv,d,bs,kv,q,how,head_scales", [
    (1, 1, 128, 16, "bf16", "bf16", "any", False),
    (2037, 8, 128, 16, "bf16", "bf16", "runs", False),
    (100, 3, 64, 32, "f32", "f32", "any", False),
    (333, 8, 128, 16, "e4m3", "bf16", "runs", False),
    (333, 5, 64, 32, "e4m3", "bf16", "runs", True),
    (61, 2, 128, 32, "e4m3", "f32", "any", False),
    (48, 1, 64, 16, "e4m3", "bf16", "any", True),
])
def test_cache_read_matches_the_pool(n, hkv, d, bs, kv, q, how, head_scales, cuda_device):
    desc, kc, vc, _, slots, (ksc, vsc), rng, g = setup(n, hkv, hkv, d, bs, kv, q, how, cuda_device, n + d,
                                                       head_scales=head_scales)
    for t in (kc, vc):  # every code and bit pattern, NaNs included
        t.view(torch.uint8).random_(0, 256, generator=g)
    slots[0] = slots[n // 2]  # a slot may come twice
    k = torch.full((n, hkv, d), 7.0, dtype=DT[q], device=cuda_device)
    v = k.clone()
    skip = torch.zeros(n, dtype=torch.bool, device=cuda_device)
    if n > 20:
        slots[5], slots[9], slots[20] = -1, desc.num_blocks * bs, -2**50
        skip[5] = skip[9] = skip[20] = True
    pa.pa_cache_read(desc, slots, kc, vc, k, v)
    torch.cuda.synchronize()
    assert bool((k[skip] == 7).all()) and bool((v[skip] == 7).all())
    ek, ev = pool_rows(desc, kc, vc, slots[~skip])
    if kv == "e4m3":
        ks = torch.full((hkv,), KS, device=cuda_device) if ksc is None else ksc
        vs = torch.full((hkv,), VS, device=cuda_device) if vsc is None else vsc
        # code * scale is one fp32 rounding, then one to the query dtype: the same in torch
        ek = (ek.view(torch.float8_e4m3fn).float() * ks[None, :, None]).to(DT[q])
        ev = (ev.view(torch.float8_e4m3fn).float() * vs[None, :, None]).to(DT[q])
    for got, exp in ((k[~skip], ek), (v[~skip], ev)):
        nan = torch.isnan(exp)
        assert torch.equal(torch.isnan(got), nan)
        if kv == "e4m3":
            assert torch.equal(got[~nan], exp[~nan])
        else:
            assert torch.equal(got.contiguous().view(torch.uint8), exp.contiguous().view(torch.uint8))


@pytest.mark.parametrize("n,hkv,d,bs,kv,q,how,head_scales", [
    (2500, 5, 128, 16, "e4m3", "bf16", "runs", True), (5000, 5, 64, 32, "e4m3", "bf16", "any", False),
    (2500, 3, 128, 32, "e4m3", "f32", "runs", False), (3001, 7, 64, 16, "e4m3", "f32", "any", True),
    (2500, 3, 128, 16, "f32", "f32", "any", False), (5003, 5, 64, 32, "bf16", "bf16", "runs", False)])
def test_cache_read_of_many_rows(n, hkv, d, bs, kv, q, how, head_scales, cuda_device):
    """Calls large enough for four vectors per thread."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert 2 * n * hkv * (d * (4 if q == "f32" else 2) // 16) > sms * 2048
    test_cache_read_matches_the_pool(n, hkv, d, bs, kv, q, how, head_scales, cuda_device)


@pytest.mark.parametrize("n", [100, 3000])
@pytest.mark.parametrize("d,kv,q", [(128, "bf16", "bf16"), (128, "e4m3", "bf16"), (64, "f32", "f32"), (64, "e4m3", "f32")])
def test_pools_past_32_bits(d, kv, q, n, cuda_device):
    """Slots whose bytes lie past 2^32 in each of the pools: written, and read back."""
    hq, hkv, bs = 8, 8, 16
    rng, g = np.random.default_rng(n), torch.Generator(device=cuda_device).manual_seed(n)
    size = {"bf16": 2, "e4m3": 1, "f32": 4}[kv]
    first, used = 2**32 // (hkv * bs * d * size) + 1, n // bs + 3
    desc = pa.CacheDesc.make(first + used, bs, hkv, hq, d, kv, q, KS, VS)
    kc, vc = pa.alloc_cache(desc, cuda_device)
    assert kc.nbytes > 2**32
    qkv = torch.randn((n, hq + 2 * hkv, d), generator=g, device=cuda_device).to(DT[q])
    xq, xk, xv = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    table = table_of(5000, d, cuda_device)
    pos = torch.from_numpy(rng.integers(0, 5000, n).astype(np.int32)).to(cuda_device)
    w = (1 + 0.3 * torch.randn(d, generator=g, device=cuda_device)).to(DT[q])
    slots = torch.from_numpy(slots_of(n, used, bs, "runs", rng)).to(cuda_device) + first * bs
    out = torch.empty((n, hq, d), dtype=DT[q], device=cuda_device)
    pa.pa_norm_rope_write(desc, pa.QkPrep.make(w, w, 1e-5, table), xq, xk, xv, pos, slots, out, kc, vc)
    close(out, fp64_rows(xq, w, 1e-5, table, pos, d, False), HALF[q])
    gk, gv = pool_rows(desc, kc, vc, slots)
    ek = fp64_rows(xk, w, 1e-5, table, pos, d, False)
    k, v = (torch.empty((n, hkv, d), dtype=DT[q], device=cuda_device) for _ in range(2))
    pa.pa_cache_read(desc, slots, kc, vc, k, v)
    if kv == "e4m3":
        close_e4m3(gk, ek, KS)
        close_e4m3(gv, xv.double(), VS)
        gk, gv = ((t.view(torch.float8_e4m3fn).float() * s).to(DT[q]) for t, s in ((gk, KS), (gv, VS)))
    else:
        close(gk, ek, HALF[q])
        assert torch.equal(gv, xv)
    assert torch.equal(k, gk) and torch.equal(v, gv)


def test_write_then_read_back(cuda_device):
    """What pa_norm_rope_write stores comes back through pa_cache_read: the run a swap-out makes."""
    desc, kc, vc, (xq, xk, xv), slots, _, rng, g = setup(200, 8, 2, 128, 16, "bf16", "bf16", "runs", cuda_device, 23)
    table = table_of(200, 128, cuda_device)
    pos = torch.arange(200, dtype=torch.int32, device=cuda_device)
    w = torch.ones(128, dtype=torch.bfloat16, device=cuda_device)
    out = torch.empty((200, 8, 128), dtype=torch.bfloat16, device=cuda_device)
    k, v = (torch.empty((200, 2, 128), dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pa.pa_norm_rope_write(desc, pa.QkPrep.make(w, w, 1e-6, table), xq, xk, xv, pos, slots, out, kc, vc)
        pa.pa_cache_read(desc, slots, kc, vc, k, v)
    side.synchronize()
    close(k, fp64_rows(xk, w, 1e-6, table, pos, 128, False), HALF["bf16"])
    assert torch.equal(v, xv)
