"""pa_decode_biased and pa_decode_chunked_prefill_biased against softmax
attention in fp64 over the same pool bytes.

Tolerance, per output element.  With p the fp64 weights, A = sum p |v|: the
weights enter P V rounded (bf16 half a step 2^-8 for a bf16 pool, f16 2^-11 for
e4m3, none in fp32), the output is rounded once (2^-8 bf16, 2^-24 fp32), and a
score's error ds moves a weight by the factor e^ds on both sides of the
division, 2 ds A in all.  ds: fp32 products and sums of D terms, at most D 2^-24
of sum |q k| scale (two MMA chains and their sum; truncating accumulation
doubles it), and a few fp32 roundings (2^-20 taken) of the score and of what the
cap and the bias add to it; fp32 sums of n weights add n 2^-24 A."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_452_b200 as pa

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
KS, VS = 0.0125, 0.011
NAN_CODE = 0x7F


class Batch:
    """A batch over a shuffled pool; what no query may see (pool slots outside the contexts, slots and table entries
    that neither prefix nor window reach) holds NaN and, for whole blocks, entries outside the pool."""

    def __init__(self, dev, qlens, lens, hq, hkv, d, bs, kv, q, cap=0.0, window=0, slopes=False, prefix=None, seed=0,
                 head_scales=False, qsize=3.0, spoil=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=dev).manual_seed(seed)
        self.qlens, self.lens = np.asarray(qlens), np.asarray(lens)
        S = len(lens)
        need = (self.lens + bs - 1) // bs
        nb = int(need.sum()) + 3
        perm = rng.permutation(nb)
        width = max(1, int(need.max()) + 1)
        tables = np.full((S, width), -7, dtype=np.int32)  # past the context: never read
        at = 0
        for s, n in enumerate(need):
            tables[s, :n] = perm[at:at + n]
            at += n
        kh = vh = None
        if head_scales:
            kh = torch.rand(hkv, generator=g, device=dev) * 0.02 + 0.005
            vh = torch.rand(hkv, generator=g, device=dev) * 0.02 + 0.005
        self.kh, self.vh = kh, vh
        self.desc = pa.CacheDesc.make(nb, bs, hkv, hq, d, kv, q, KS, VS, kh, vh)
        self.prefix = None if prefix is None else np.asarray(prefix)
        pfx = np.zeros(S, dtype=np.int64) if prefix is None else np.clip(self.prefix, 0, self.lens)
        self.window, self.cap, self.scale = window, cap, 1 / math.sqrt(d)
        shape = (nb, hkv, bs, d)
        if kv == "e4m3":
            k = (torch.randn(shape, generator=g, device=dev) / KS).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            v = (torch.randn(shape, generator=g, device=dev) / VS).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            k, v = (torch.randn(shape, generator=g, device=dev).to(DT[kv]) for _ in range(2))
        bad = NAN_CODE if kv == "e4m3" else float("nan")
        seen = torch.zeros((nb, bs), dtype=torch.bool)
        for s in range(S):
            lo = max(0, int(self.lens[s] - self.qlens[s] - window + 1)) if window and self.qlens[s] else 0
            for j in range(int(self.lens[s])):
                if self.qlens[s] and (j < pfx[s] or j >= lo):
                    seen[tables[s, j // bs], j % bs] = True
        self.k_ok, self.v_ok = k.clone(), v.clone()
        if spoil:
            hidden = (~seen).to(dev)
            k.transpose(1, 2)[hidden] = bad
            v.transpose(1, 2)[hidden] = bad
        self.tables_ok = torch.from_numpy(np.maximum(tables, 0)).to(dev)
        if spoil and window:
            for s in range(S):
                np_, wb = -(-int(pfx[s]) // bs), max(0, int(self.lens[s] - self.qlens[s] - window + 1)) // bs
                tables[s, np_:max(np_, wb)] = nb + 5  # freed: outside the pool
        self.k, self.v = k, v.transpose(2, 3).contiguous() if kv == "e4m3" else v
        self.tables = torch.from_numpy(tables).to(dev)
        rows = int(self.qlens.sum())
        self.q = (qsize * torch.randn((rows, hq, d), generator=g, device=dev)).to(DT[q])
        self.slopes = (torch.from_numpy((2.0 ** (-8.0 * (np.arange(hq) + 1) / hq)).astype(np.float32)).to(dev)
                       if slopes else None)
        self.qsl = torch.from_numpy(np.concatenate([[0], np.cumsum(self.qlens)]).astype(np.int32)).to(dev)
        self.sl = torch.from_numpy(self.lens.astype(np.int32)).to(dev)
        self.mod = pa.ScoreMod.make(cap, window, self.slopes,
                                    None if prefix is None else torch.from_numpy(self.prefix.astype(np.int32)).to(dev))
        self.out = torch.full((rows, hq, d), float("nan"), dtype=DT[q], device=dev)
        self.ws = pa.alloc_workspace(pa.pa_biased_workspace_size(self.desc, S, rows), dev)
        self.kv, self.qd, self.pfx = kv, q, pfx

    def run(self, decode=None, stream=None):
        d = self.desc
        if decode if decode is not None else bool((self.qlens == 1).all()):
            pa.pa_decode_biased(d, self.mod, self.q, self.k, self.v, self.tables, self.sl, self.scale, self.out, self.ws,
                                stream)
        else:
            pa.pa_decode_chunked_prefill_biased(d, self.mod, self.q, self.k, self.v, self.tables, self.qsl, self.sl,
                                                int(self.qlens.max()), self.scale, self.out, self.ws, stream)

    def expected(self):
        """fp64 outputs and the tolerance of every element."""
        d, hkv, hq, bs = self.desc.head_dim, self.desc.num_kv_heads, self.desc.num_q_heads, self.desc.block_size
        out = torch.zeros(self.out.shape, dtype=torch.float64, device=self.out.device)
        tol = torch.full_like(out, 1e-7)
        val = lambda t: (t.view(torch.float8_e4m3fn) if self.kv == "e4m3" else t).double()  # noqa: E731
        prow = {"f32": 0.0, "bf16": 2.0**-8, "e4m3": 2.0**-11 if self.qd == "bf16" else 0.0}[self.kv]
        orow = 2.0**-8 if self.qd == "bf16" else 2.0**-24
        for s in range(len(self.lens)):
            n, r = int(self.lens[s]), int(self.qlens[s])
            if n == 0 or r == 0:
                continue
            t = self.tables_ok[s, :(n + bs - 1) // bs].long()
            one = torch.ones(hkv, device=out.device, dtype=torch.float64)
            ks = one if self.kv != "e4m3" else (self.kh.double() if self.kh is not None else one * float(np.float32(KS)))
            vs = one if self.kv != "e4m3" else (self.vh.double() if self.vh is not None else one * float(np.float32(VS)))
            k = val(self.k_ok[t]).transpose(0, 1).reshape(hkv, -1, d)[:, :n] * ks[:, None, None]
            v = val(self.v_ok[t]).transpose(0, 1).reshape(hkv, -1, d)[:, :n] * vs[:, None, None]
            i = torch.arange(n - r, n, device=out.device)[:, None]
            j = torch.arange(n, device=out.device)[None]
            see = j <= i
            if self.window:
                see = see & (i - j < self.window)
            see = see | (j < int(self.pfx[s]))
            a, b = int(self.qsl[s]), int(self.qsl[s + 1])
            for h in range(hq):
                kk, vv = k[h * hkv // hq], v[h * hkv // hq]
                q = self.q[a:b, h].double()
                x = q @ kk.T * self.scale
                size = (q.abs() @ kk.abs().T * self.scale).masked_fill(~see, 0)
                y = self.cap * torch.tanh(x / self.cap) if self.cap else x
                bias = float(self.slopes[h]) * (i - j).abs() if self.slopes is not None else torch.zeros_like(x)
                p = torch.softmax((y - bias).masked_fill(~see, -math.inf), -1)
                out[a:b, h] = p @ vv
                some = see & (p > 1e-9)
                ds = (2 * d * 2.0**-24 * size.masked_fill(~some, 0)
                      + 2.0**-20 * (y.abs() + bias + self.cap).masked_fill(~some, 0)).amax(-1, keepdim=True) + 2.0**-20
                A = p @ vv.abs()
                tol[a:b, h] = (prow + 2 * ds + n * 2.0**-24) * A + orow * out[a:b, h].abs() + 1e-7
        return out, tol

    def check(self):
        torch.cuda.synchronize()
        assert pa.workspace_error(self.ws) == 0
        exp, tol = self.expected()
        got = self.out.double()
        assert bool(torch.isfinite(got).all())
        over = (got - exp).abs() / tol
        assert float(over.max()) <= 1, (float(over.max()), float((got - exp).abs().max()))


LENS = [1, 2, 15, 16, 17, 31, 33, 64, 100, 129, 300, 517]
MODS = [dict(), dict(cap=30.0), dict(window=1), dict(window=40), dict(window=129, slopes=True),
        dict(slopes=True), dict(cap=50.0, slopes=True, window=77, prefix="some"), dict(prefix="some", window=16)]


def prefix_of(mod, lens):
    if mod.get("prefix") != "some":
        return mod
    return {**mod, "prefix": [[0, 3, 16, 40, 1000, -5][i % 6] for i in range(len(lens))]}


@pytest.mark.parametrize("mod", MODS, ids=str)
@pytest.mark.parametrize("hq,hkv,d,bs,kv,q", [
    (8, 2, 128, 16, "bf16", "bf16"), (3, 3, 64, 32, "bf16", "bf16"), (16, 1, 128, 32, "bf16", "bf16"),
    (12, 2, 64, 16, "e4m3", "bf16"), (8, 1, 128, 16, "e4m3", "bf16"), (11, 1, 128, 32, "e4m3", "bf16"),
    (4, 2, 64, 16, "f32", "f32"), (3, 1, 128, 32, "e4m3", "f32")])
def test_decode_matches_fp64(hq, hkv, d, bs, kv, q, mod, cuda_device):
    lens = LENS + [0]
    b = Batch(cuda_device, [1] * len(lens), lens, hq, hkv, d, bs, kv, q, **prefix_of(mod, lens), seed=d + hq,
              head_scales=kv == "e4m3" and hq == 8)
    b.run(decode=True)
    b.check()
    assert bool((b.out[-1] == 0).all())  # an empty context: a zero row
    first = b.out.clone()
    b.out.fill_(5)
    b.run(decode=True)  # again over the same workspace: the same bits
    torch.cuda.synchronize()
    assert torch.equal(first, b.out)


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("e4m3", 64)])
def test_decode_long_contexts(kv, d, cuda_device):
    """Contexts cut over many warps, with and without a gap between prefix and window."""
    for mod in (dict(cap=20.0, slopes=True), dict(window=3000, prefix=[100, 0, 9000])):
        b = Batch(cuda_device, [1, 1, 1], [9001, 20000, 9000], 8, 2, d, 16, kv, "bf16", **mod, seed=5)
        b.run(decode=True)
        b.check()


CHUNKS = [([5], [5]), ([33], [133]), ([128, 1, 0, 130, 64, 1, 2], [128, 77, 50, 400, 1000, 1, 2]),
          ([300, 257], [300, 900]), ([2], [700])]


@pytest.mark.parametrize("mod", MODS, ids=str)
@pytest.mark.parametrize("shape", range(len(CHUNKS)))
@pytest.mark.parametrize("hq,hkv,d,bs,kv,q", [
    (8, 2, 128, 16, "bf16", "bf16"), (3, 3, 64, 32, "bf16", "bf16"), (6, 1, 128, 32, "bf16", "bf16"),
    (16, 2, 64, 16, "bf16", "bf16"), (8, 2, 128, 16, "e4m3", "bf16"), (5, 1, 64, 32, "e4m3", "bf16"),
    (4, 2, 64, 16, "f32", "f32"), (3, 1, 128, 32, "e4m3", "f32")])
def test_chunks_match_fp64(hq, hkv, d, bs, kv, q, shape, mod, cuda_device):
    qlens, lens = CHUNKS[shape]
    b = Batch(cuda_device, qlens, lens, hq, hkv, d, bs, kv, q, **prefix_of(mod, lens), seed=d + hq + shape,
              head_scales=kv == "e4m3" and hq == 8)
    b.run(decode=False)
    b.check()
    first = b.out.clone()
    b.out.fill_(5)
    b.run(decode=False)
    torch.cuda.synchronize()
    assert torch.equal(first, b.out)


@pytest.mark.parametrize("mod", [dict(), dict(cap=30.0, slopes=True), dict(window=700, prefix=[300, 0, 2500, 0]),
                                 dict(slopes=True, prefix=[4000, 129, 1, 0])], ids=str)
@pytest.mark.parametrize("hq,hkv,d,bs,kv", [(8, 2, 128, 16, "bf16"), (1, 1, 64, 32, "bf16"), (8, 1, 128, 32, "e4m3"),
                                            (6, 2, 64, 16, "e4m3")])
def test_few_rows_over_long_contexts(hq, hkv, d, bs, kv, mod, cuda_device):
    """Few units: their keys are cut over several SMs and joined; short ones beside long ones have fewer parts."""
    b = Batch(cuda_device, [16, 2, 70, 1], [4000, 130, 2500, 3000], hq, hkv, d, bs, kv, "bf16", **mod, seed=d)
    for _ in range(3):  # the counters start every call at zero
        b.out.fill_(float("nan"))
        b.run(decode=False)
        b.check()


@pytest.mark.parametrize("mod", [dict(cap=30.0), dict(window=77, prefix="some", slopes=True)], ids=str)
@pytest.mark.parametrize("hq,hkv,d,bs,kv", [(8, 2, 128, 16, "f32"), (6, 2, 64, 32, "f32"), (16, 1, 128, 32, "e4m3"),
                                            (8, 8, 64, 16, "e4m3")])
def test_fp32_chunks_in_tiles(hq, hkv, d, bs, kv, mod, cuda_device):
    """fp32 chunks with rows enough for the tile kernel, a single row and an empty sequence among them."""
    lens = [400, 9, 300, 65]
    b = Batch(cuda_device, [290, 0, 100, 1], lens, hq, hkv, d, bs, kv, "f32", **prefix_of(mod, lens), seed=d,
              head_scales=kv == "e4m3")
    assert 391 * hq >= 2048
    b.run(decode=False)
    b.check()


@pytest.mark.parametrize("kv", ["f32", "e4m3"])
@pytest.mark.parametrize("qlens", [[1] * 30 + [2] + [1] * 32, [1] * 30 + [70] + [1] * 32, [0] * 90 + [80] + [0] * 30],
                         ids=["a short chunk", "a long chunk", "empty sequences"])
def test_fp32_chunks_among_single_rows(qlens, kv, cuda_device):
    """fp32: many single rows beside one chunk, and a chunk among empty sequences."""
    rng = np.random.default_rng(16)
    lens = [q + int(rng.integers(0, 300)) for q in qlens]
    b = Batch(cuda_device, qlens, lens, 32, 4, 64, 16, kv, "f32", cap=30.0, slopes=True, seed=16)
    b.run(decode=False)
    b.check()


def test_many_chunks(cuda_device):
    """More chunks than are put in order, between decode rows and empty sequences."""
    rng = np.random.default_rng(2)
    qlens = [int(rng.choice([0, 1, 1, 2, 5, 40])) for _ in range(300)]
    lens = [q + int(rng.integers(0, 200)) if q else 7 for q in qlens]
    b = Batch(cuda_device, qlens, lens, 4, 2, 64, 16, "bf16", "bf16", cap=20.0, window=50, seed=2)
    b.run(decode=False)
    b.check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_many_units_per_sm(kv, cuda_device):
    """Every CTA takes its queue entries many times over: 330 two-row chunks of 32 kv heads."""
    rng = np.random.default_rng(4)
    lens = [int(n) for n in rng.integers(2, 60, 330)]
    b = Batch(cuda_device, [2] * 330, lens, 32, 32, 64, 16, kv, "bf16", cap=20.0, seed=4, spoil=False)
    b.run(decode=False)
    b.check()


def test_rows_of_others_stay(cuda_device):
    """A row past the last sequence's, as in a padded batch, keeps what it held."""
    for kv in ("bf16", "e4m3"):
        b = Batch(cuda_device, [40, 1, 3], [90, 33, 200], 8, 2, 128, 16, kv, "bf16", cap=30.0, seed=5)
        pad = 9
        q, out = b.q, b.out
        b.q = torch.cat([q, torch.full((pad, 8, 128), float("nan"), dtype=q.dtype, device=cuda_device)])
        b.out = torch.full((q.shape[0] + pad, 8, 128), 3.0, dtype=q.dtype, device=cuda_device)
        b.run(decode=False)
        torch.cuda.synchronize()
        assert bool((b.out[-pad:] == 3).all())
        b.q, b.out = q, b.out[:-pad].contiguous()
        b.check()


@pytest.mark.parametrize("kv,q", [("bf16", "bf16"), ("e4m3", "bf16"), ("f32", "f32"), ("e4m3", "f32")])
def test_padding_that_looks_like_full_chunks(kv, q, cuda_device):
    """num_seqs * max_q_len rows of which the last lie past every sequence's: the single rows are still computed."""
    b = Batch(cuda_device, [1, 7, 1, 0], [90, 33, 200, 12], 8, 2, 64, 16, kv, q, cap=30.0, window=50, seed=6)
    rows, full = b.q.shape[0], 28
    kept = b.q
    b.q = torch.cat([kept, torch.full((full - rows, 8, 64), float("nan"), dtype=kept.dtype, device=cuda_device)])
    b.out = torch.full((full, 8, 64), 3.0, dtype=kept.dtype, device=cuda_device)
    b.ws = pa.alloc_workspace(pa.pa_biased_workspace_size(b.desc, 4, full), cuda_device)
    b.run(decode=False)
    torch.cuda.synchronize()
    assert bool((b.out[rows:] == 3).all())
    b.q, b.out = kept, b.out[:rows].contiguous()
    b.check()


@pytest.mark.parametrize("kv,q,hq", [("bf16", "bf16", 8), ("e4m3", "bf16", 8), ("f32", "f32", 8), ("f32", "f32", 2)])
@pytest.mark.parametrize("rows", [1, 200, 362])
def test_rows_past_the_queries_are_left_out(rows, kv, q, hq, cuda_device):
    """query_start_loc that goes on past the rows of q and out (a step cut to fewer rows): the rows there are are right,
    what lies behind them stays.  The cut falls behind a single row, inside the first chunk and before the last single
    rows, one of them with an empty context; the buffers go on behind the cut."""
    b = Batch(cuda_device, [1, 260, 1, 100, 1, 1], [90, 333, 40, 100, 200, 0], hq, 2, 64, 16, kv, q, cap=30.0, window=150,
              seed=13)
    exp, tol = b.expected()
    whole = torch.full_like(b.out, 3.0)
    b.q, b.out = b.q[:rows], whole[:rows]
    b.run(decode=False)
    torch.cuda.synchronize()
    assert pa.workspace_error(b.ws) == 0
    assert bool((whole[rows:] == 3).all())
    assert bool(((b.out.double() - exp[:rows]).abs() <= tol[:rows]).all())


@pytest.mark.parametrize("kv,q", [("bf16", "bf16"), ("e4m3", "bf16"), ("f32", "f32")])
def test_a_window_past_every_context(kv, q, cuda_device):
    """The largest window hides nothing, whatever the prefix: its arithmetic does not wrap."""
    b = Batch(cuda_device, [1, 300, 1, 70], [900, 1300, 64, 70], 8, 2, 64, 16, kv, q, window=2**31 - 1,
              prefix=[1000, 1300, 0, 33], slopes=True, seed=7)
    b.run(decode=False)
    b.check()


def test_capped_fp32_keeps_fp32(cuda_device):
    """The cap in fp32 rows: within 1e-5 of the fp64 result in the 2-norm."""
    b = Batch(cuda_device, [1] * 5, [40, 128, 300, 64, 511], 4, 2, 64, 16, "f32", "f32", cap=50.0, slopes=True, seed=1)
    b.run(decode=True)
    exp, _ = b.expected()
    assert float((b.out.double() - exp).norm() / exp.norm()) < 1e-5


def test_decode_behind_a_chunk_on_the_same_output(cuda_device):
    """Calls follow one another on one stream without a gap and over one output: a decode step right behind a chunk
    step that writes the same rows, its empty contexts' zero rows included."""
    big = Batch(cuda_device, [512, 512], [3000, 3500], 8, 2, 128, 16, "bf16", "bf16", cap=30.0, seed=1)
    small = Batch(cuda_device, [1] * 6, [0, 40, 0, 900, 0, 17], 8, 2, 128, 16, "bf16", "bf16", cap=30.0, seed=2)
    for _ in range(5):
        small.out = big.out[:6]
        big.run(decode=False)
        small.run(decode=True)
        torch.cuda.synchronize()
        small.check()
        assert bool((small.out[[0, 2, 4]] == 0).all())


@pytest.mark.parametrize("bs", [16, 32])
def test_mixed_steps_back_to_back(bs, cuda_device):
    """Mixed steps of different sizes over one workspace, without a gap: each one's chunks run beside its single rows
    and partly behind them, and its results stay the same bits."""
    big = Batch(cuda_device, [300, 1, 1, 200, 1, 1, 1, 450], [900, 3000, 40, 1500, 2, 700, 5, 450], 16, 4, 128, bs, "bf16",
                "bf16", cap=40.0, window=800, prefix=[16] * 8, seed=1)
    many = Batch(cuda_device, [1] * 90 + [70] + [1] * 60, list(range(7, 157 * 9, 9))[:151], 8, 2, 64, bs, "bf16", "bf16",
                 slopes=True, seed=2)
    none = Batch(cuda_device, [3, 5, 0, 4], [60, 5, 9, 400], 8, 2, 128, bs, "bf16", "bf16", cap=9.0, seed=3)
    rows = Batch(cuda_device, [1] * 7, [5000, 1, 0, 4000, 300, 9000, 17], 32, 2, 64, bs, "bf16", "bf16", cap=9.0, seed=4)
    codes = Batch(cuda_device, [1, 1, 90], [6000, 2500, 90], 8, 1, 128, bs, "e4m3", "bf16", slopes=True, seed=5)
    batches = (big, many, none, rows, codes)
    ws = max((b.ws for b in batches), key=lambda t: t.numel())
    first = []
    for b in batches:
        b.ws = ws
        b.run(decode=False)
        b.check()
        first.append(b.out.clone())
        b.out.zero_()
    for _ in range(20):
        for b in batches:
            b.run(decode=False)
    torch.cuda.synchronize()
    for b, was in zip(batches, first):
        assert torch.equal(b.out, was)
        b.check()


@pytest.mark.parametrize("bs", [16, 32])
def test_many_single_rows_beside_chunks(bs, cuda_device):
    """Enough single rows that chunks start before them: every row is right, and again the same bits when the step is
    repeated without a gap, captured, and followed by a step without chunks."""
    rng = np.random.default_rng(bs)
    qlens = [1] * 70
    lens = [int(n) for n in rng.integers(1, 900, 70)]
    for s, n in ((3, 260), (40, 33), (69, 500)):
        qlens[s], lens[s] = n, n + 77 * s
    b = Batch(cuda_device, qlens, lens, 16, 8, 128, bs, "bf16", "bf16", cap=30.0, window=700, prefix=[9] * 70, seed=bs)
    one = Batch(cuda_device, [1] * 70, lens, 16, 8, 128, bs, "bf16", "bf16", cap=30.0, seed=bs + 1)
    b.run(decode=False)
    b.check()
    was = b.out.clone()
    b.out.zero_()
    for _ in range(15):
        b.run(decode=False)
        one.run(decode=True)
    torch.cuda.synchronize()
    assert torch.equal(b.out, was)
    one.check()
    b.out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            b.run(decode=False)
            b.run(decode=False)
        g.replay()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, was)
    b.check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_cut_units_of_many_chunks(kv, cuda_device):
    """More chunks than are taken in order, but few enough units that their keys are cut."""
    lens = [2 + 11 * s for s in range(70)]
    b = Batch(cuda_device, [2] * 70, lens, 4, 1, 64, 16, kv, "bf16", cap=20.0, window=400, prefix=[20] * 70, seed=11)
    b.run(decode=False)
    b.check()
    was = b.out.clone()
    b.run(decode=False)
    b.check()
    assert torch.equal(b.out, was)


@pytest.mark.parametrize("group", [17, 65, 127, 131, 256])
@pytest.mark.parametrize("kv,q", [("bf16", "bf16"), ("e4m3", "bf16"), ("f32", "f32")])
def test_large_groups(group, kv, q, cuda_device):
    """Groups past a query tile's rows or with no divisor that fits, in chunks and single rows."""
    b = Batch(cuda_device, [1, 9, 0, 1, 40], [30, 200, 5, 700, 64], group, 1, 64, 16, kv, q, cap=20.0, window=60,
              slopes=True, prefix=[4] * 5, seed=group)
    b.run(decode=False)
    b.check()


def test_scalars_as_the_plain_calls_take_them(cuda_device):
    """A scale and a max_q_len that are tensors of one element."""
    b = Batch(cuda_device, [3, 1], [40, 90], 8, 2, 64, 16, "bf16", "bf16", seed=3)
    b.scale = torch.tensor(b.scale, dtype=torch.float64)
    pa.pa_decode_chunked_prefill_biased(b.desc, b.mod, b.q, b.k, b.v, b.tables, b.qsl, b.sl, torch.tensor(3), b.scale,
                                        b.out, b.ws)
    b.scale = float(b.scale)
    b.check()


def test_a_group_of_more_than_128(cuda_device):
    b = Batch(cuda_device, [3, 1], [40, 90], 130, 1, 64, 16, "bf16", "bf16", cap=10.0, seed=3)
    b.run(decode=False)
    b.check()


def test_scores_that_fill_the_cap(cuda_device):
    """Scores far past the cap on both sides: tanh saturates, nothing overflows."""
    for kv in ("bf16", "e4m3"):
        b = Batch(cuda_device, [70, 1], [200, 90], 8, 2, 128, 16, kv, "bf16", cap=5.0, seed=9, qsize=60.0)
        b.run(decode=False)
        b.check()


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("size", [2.0**-60, 2.0**-30, 2.0**14, 2.0**20, 2.0**100])
def test_queries_past_the_range_of_f16(size, cap, cuda_device):
    """bf16 queries that f16 cannot hold, with a scale that brings their scores back: an e4m3 pool's products take them
    as they are (a power of two changes nothing else in the arithmetic)."""
    for qlens, lens in (([1] * 4, [300, 17, 64, 900]), ([70, 1, 130], [200, 90, 130])):
        b = Batch(cuda_device, qlens, lens, 12, 2, 128, 16, "e4m3", "bf16", cap=cap, seed=14)
        b.q, b.scale = (b.q.float() * size).to(torch.bfloat16), b.scale / size
        b.run()
        b.check()


def test_queries_of_many_sizes_in_a_group(cuda_device):
    """Heads of one group whose queries differ by powers of two, a row of zeros among them: every row by its own."""
    for qlens, lens in (([1] * 3, [300, 17, 900]), ([70, 1, 20], [200, 90, 130])):
        b = Batch(cuda_device, qlens, lens, 8, 1, 64, 32, "e4m3", "bf16", cap=0.0, slopes=True, seed=15)
        size = 2.0 ** torch.tensor([0, -40, 1, -20, 0, 2, -100, 0], device=cuda_device)
        b.q = (b.q.float() * size[None, :, None]).to(torch.bfloat16)
        b.q[:, 4] = 0
        b.run()
        b.check()


def test_without_mod_as_plain_attention(cuda_device):
    """With nothing set the biased decode computes what pa_decode does.  The two cut contexts into different pieces,
    and a weight is rounded to bf16 relative to its piece's reference, so a weight may differ by two roundings of
    2^-9 and a result by two of its own: each of the two is within the tolerance of the fp64 result, which counts
    2^-8 per weight and per result, and so within twice that of the other."""
    b = Batch(cuda_device, [1] * 12, LENS, 8, 2, 128, 16, "bf16", "bf16", seed=4, spoil=False)
    b.run(decode=True)
    out = torch.empty_like(b.out)
    ws = pa.alloc_workspace(pa.pa_decode_workspace_size(b.desc, 12), cuda_device)
    pa.pa_decode(b.desc, b.q, b.k, b.v, b.tables, b.sl, b.scale, out, ws)
    b.check()
    _, tol = b.expected()
    assert bool(((out.double() - b.out.double()).abs() <= 2 * tol).all())


def test_bad_table_entries_and_long_contexts_are_flagged(cuda_device):
    for qlens in ([1, 1], [40, 1]):
        b = Batch(cuda_device, qlens, [100, 60], 8, 2, 128, 16, "bf16", "bf16", cap=30.0, seed=6, spoil=False)
        b.tables[0, 2] = b.desc.num_blocks
        b.run(decode=False)
        torch.cuda.synchronize()
        assert pa.workspace_error(b.ws) == 2
        exp, tol = b.expected()
        last = (b.out[-1].double() - exp[-1]).abs() <= tol[-1]
        assert bool(last.all())  # the other sequence is not touched by it
        b.ws.zero_()
        b.tables[0, 2] = 0
        b.sl[0] = 16 * b.tables.shape[1] + 1
        b.run(decode=False)
        torch.cuda.synchronize()
        assert pa.workspace_error(b.ws) == 3


@pytest.mark.parametrize("qlens,lens", [([1] * 3, [300, 17, 900]), ([70, 1, 130], [200, 90, 130])], ids=["decode", "chunks"])
@pytest.mark.parametrize("hq,hkv,d,kv,q", [(8, 8, 128, "bf16", "bf16"), (8, 4, 128, "e4m3", "bf16"),
                                           (8, 8, 64, "e4m3", "bf16"), (8, 8, 64, "f32", "f32"),
                                           (32, 8, 128, "e4m3", "f32")])
def test_pools_past_32_bits(hq, hkv, d, kv, q, qlens, lens, cuda_device):
    """Blocks whose bytes lie past 2^32 in each of the pools."""
    b = Batch(cuda_device, qlens, lens, hq, hkv, d, 16, kv, q, cap=30.0, slopes=True, seed=18, spoil=False)
    bytes_per_block = b.k[0].nbytes
    blocks = 2**32 // bytes_per_block + b.desc.num_blocks + 1
    first = blocks - b.desc.num_blocks
    far = []
    for t in (b.k, b.v):
        far.append(torch.empty((blocks, *t.shape[1:]), dtype=t.dtype, device=cuda_device))
        far[-1][first:] = t
    b.k, b.v = far
    b.tables = torch.where(b.tables >= 0, b.tables + first, b.tables)
    b.desc = pa.CacheDesc.make(blocks, 16, hkv, hq, d, kv, q, KS, VS)
    b.run()
    b.check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("which", ["pa_decode_biased", "pa_decode_chunked_prefill_biased", "pa_decode"])
def test_first_call_of_a_host_thread(which, kv, cuda_device):
    """A call from a host thread that has made no CUDA call of its own (no context is bound to it yet), over pools and
    queries whose maps are not known from an earlier call."""
    import threading
    qlens = [40, 1] if which == "pa_decode_chunked_prefill_biased" else [1, 1]
    b = Batch(cuda_device, qlens, [200, 300], 8, 2, 128, 16, kv, "bf16", seed=17, spoil=False)
    if which == "pa_decode":
        b.ws = pa.alloc_workspace(pa.pa_decode_workspace_size(b.desc, 2), cuda_device)
    stream, failed = torch.cuda.current_stream().cuda_stream, []

    def call():
        try:
            if which == "pa_decode":
                pa.pa_decode(b.desc, b.q, b.k, b.v, b.tables, b.sl, b.scale, b.out, b.ws, stream)
            else:
                b.run(stream=stream)
        except pa.PaError as e:
            failed.append(str(e))
    t = threading.Thread(target=call)
    t.start()
    t.join()
    assert not failed
    b.check()


def test_host_threads_call_at_once(cuda_device):
    """Host threads that call with batches of other sizes (other shared-memory sizes of one kernel) on one stream."""
    from concurrent.futures import ThreadPoolExecutor
    batches = [Batch(cuda_device, [1] * n, [1 + (37 * i + 11 * n) % 900 for i in range(n)], 8, 2, 128, 16, "bf16", "bf16",
                     cap=30.0, seed=n, spoil=False) for n in (3, 60, 700, 1500)]
    stream = torch.cuda.current_stream()

    def calls(b):
        for _ in range(60):
            b.run(decode=True, stream=stream)
    with ThreadPoolExecutor(len(batches)) as pool:
        list(pool.map(calls, batches))
    for b in batches:
        b.check()


def test_captured_and_replayed(cuda_device):
    """A mixed step captured into a graph and replayed on other inputs."""
    b = Batch(cuda_device, [40, 1, 1], [200, 300, 17], 8, 2, 128, 16, "bf16", "bf16", cap=30.0, window=60, seed=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run(decode=False)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(decode=False)
    for i in range(3):
        b.q.copy_(torch.randn(b.q.shape, device=cuda_device) * 2)
        b.out.fill_(float("nan"))
        g.replay()
        b.check()
    del g


def test_a_layer_step(cuda_device):
    """Norm, rotation and write, then the biased attention and the read-back, as a layer runs them."""
    hq, hkv, d, bs, n = 8, 2, 128, 16, 90
    b = Batch(cuda_device, [n], [n], hq, hkv, d, bs, "bf16", "bf16", cap=30.0, window=50, seed=12, spoil=False)
    g = torch.Generator(device=cuda_device).manual_seed(1)
    qkv = torch.randn((n, hq + 2 * hkv, d), generator=g, device=cuda_device).to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(d, generator=g, device=cuda_device)).to(torch.bfloat16)
    ang = torch.arange(n, device=cuda_device)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, device=cuda_device) / d)[None]
    prep = pa.QkPrep.make(w, w, 1e-6, torch.cat([ang.cos(), ang.sin()], 1).float())
    pos = torch.arange(n, dtype=torch.int32, device=cuda_device)
    slots = b.tables_ok[0].long()[pos.long() // bs] * bs + pos.long() % bs
    pa.pa_norm_rope_write(b.desc, prep, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, slots, b.q, b.k, b.v)
    b.run(decode=False)
    k, v = (torch.empty((n, hkv, d), dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    pa.pa_cache_read(b.desc, slots, b.k, b.v, k, v)
    b.k_ok, b.v_ok = b.k, b.v
    b.check()
    assert torch.equal(v, qkv[:, hq + hkv:])
    assert torch.equal(k, b.k[slots // bs, :, slots % bs])
