"""Measured cases of the layer-step operators around the paged cache: norms and
rotation of queries and keys with the cache write, reading the cache back, and
attention with a capped or distance-biased score, a sliding window and an
always-visible prefix, for single tokens and for chunks of new tokens.

``run`` computes an operator in plain torch operations (``own`` false) or by
the library's calls (``own`` true); ``exact`` computes it in 64 bits."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
K_SCALE, V_SCALE = 0.0125, 0.011  # e4m3 pools: N(0, 1) rows fill the code range up to about 5 sigma


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 sequences, one layer: latency counts
        dict(name="prep_decode_64", op="prep", tokens=64, hq=32, hkv=8, d=128, bs=16, kv="bf16", q="bf16", rot=128,
             inter=False, positions=4096),
        # a mixed step: 8 chunks of 512 tokens and 248 decode tokens
        dict(name="prep_step_4344", op="prep", tokens=4344, hq=32, hkv=8, d=128, bs=16, kv="bf16", q="bf16", rot=128,
             inter=False, positions=8192),
        # long prompts of a 64-head model written into a quantised pool
        dict(name="prep_long_e4m3", op="prep", tokens=16384, hq=64, hkv=8, d=128, bs=16, kv="e4m3", q="bf16", rot=128,
             inter=False, positions=32768),
        # one sequence's cache read back (swapped out, or checked)
        dict(name="read_one_bf16", op="read", tokens=2037, hq=32, hkv=8, d=128, bs=16, kv="bf16", q="bf16"),
        # a batch of long contexts read back from a quantised pool
        dict(name="read_long_e4m3", op="read", tokens=131072, hq=64, hkv=8, d=128, bs=16, kv="e4m3", q="bf16"),
        # the smallest decode step: 4 short sequences, fp32, a bias per distance
        dict(name="decode_tiny_f32", op="decode", seqs=4, lo=40, hi=300, hq=2, hkv=2, d=64, bs=16, kv="f32", q="f32",
             cap=0.0, window=0, slopes=True, prefix=0),
        # a decode batch of a model with capped scores and a sliding window
        dict(name="decode_cap_window", op="decode", seqs=64, lo=32, hi=2048, hq=32, hkv=8, d=128, bs=16, kv="bf16",
             q="bf16", cap=50.0, window=1024, slopes=False, prefix=16),
        # long contexts over a quantised pool with a bias per distance
        dict(name="decode_long_e4m3", op="decode", seqs=32, lo=4096, hi=32768, hq=64, hkv=8, d=128, bs=16, kv="e4m3",
             q="bf16", cap=0.0, window=0, slopes=True, prefix=0),
        # a short prompt's last chunk, alone in its step
        dict(name="chunk_small_cap", op="chunk", chunks=1, rows=33, prior=100, decodes=0, hi=0, hq=8, hkv=2, d=64, bs=16,
             kv="bf16", q="bf16", cap=30.0, window=0, slopes=False, prefix=0),
        # a mixed step: 8 chunks of 512 over up to 4096 cached tokens and 248 decode rows, capped, windowed
        dict(name="chunk_mixed_cap", op="chunk", chunks=8, rows=512, prior=4096, decodes=248, hi=4096, hq=32, hkv=8, d=128,
             bs=16, kv="bf16", q="bf16", cap=50.0, window=2048, slopes=False, prefix=0),
        # prompts whose first 512 tokens see one another both ways, a bias per distance, one head per kv head
        dict(name="chunk_prefix_slopes", op="chunk", chunks=6, rows=640, prior=2048, decodes=0, hi=0, hq=32, hkv=32, d=128,
             bs=16, kv="bf16", q="bf16", cap=0.0, window=0, slopes=True, prefix=512),
        # chunks of long prompts over a quantised pool
        dict(name="chunk_long_e4m3", op="chunk", chunks=2, rows=1024, prior=8192, decodes=0, hi=0, hq=32, hkv=8, d=128,
             bs=16, kv="e4m3", q="bf16", cap=50.0, window=0, slopes=False, prefix=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prep", "read", "decode", "decode", "chunk", "chunk"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 4, 6, 8, 16 if hkv <= 4 else 5])
    c = dict(op=op, hq=hkv * g, hkv=hkv, d=d, bs=rng.choice([16, 32]))
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    q = "bf16"
    if op == "prep":
        if rng.random() < 0.2:
            q, kv = "f32", rng.choice(["f32", "e4m3"])
        c.update(tokens=_log(rng, 1, 16384), positions=_log(rng, 2048, 131072), rot=rng.choice([d, d, d // 2, d // 4]),
                 inter=rng.random() < 0.3)
    elif op == "read":
        if rng.random() < 0.2:
            q, kv = "f32", rng.choice(["f32", "e4m3"])
        c.update(tokens=_log(rng, 1, 131072 if q == "bf16" else 65536))
    else:
        small = op == "decode" and rng.random() < 0.2
        if small:
            q = kv = "f32"
        c.update(cap=rng.choice([0.0, 20.0, 30.0, 50.0]), slopes=rng.random() < 0.5,
                 window=rng.choice([0, 0, 1]) and _log(rng, 33, 4096), prefix=rng.choice([0, 0, 4, 129]))
        if op == "decode":
            hi = _log(rng, 64, 512 if small else 16384)
            c.update(seqs=_log(rng, 1, max(1, min(64, 262144 // hi))), lo=max(1, hi // 8), hi=hi)
        else:
            rows = _log(rng, 2, 1024)
            c.update(chunks=rng.randint(1, max(1, min(8, 2048 // rows))), rows=rows, prior=_log(rng, 1, 4096 if hkv * g <= 32 else 1024),
                     decodes=rng.choice([0, 0, rng.randint(1, 64)]), hi=1000)
    c.update(kv=kv, q=q)
    return c


# ---- inputs -------------------------------------------------------------------

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _pools(case, blocks, g):
    """K pool [NB][Hkv][bs][D]; V pool the same, d-major [NB][Hkv][D][bs] for e4m3."""
    shape = (blocks, case["hkv"], case["bs"], case["d"])
    def one(scale, flip):
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if case["kv"] == "f32" else torch.bfloat16)
        if case["kv"] != "e4m3":
            return x
        x = (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return x.transpose(2, 3).contiguous() if flip else x
    return one(K_SCALE, False), one(V_SCALE, True)


def _tables(lens, bs, rng):
    """A shuffled pool of 1.25 times the blocks needed, and the sequences' tables."""
    need = (lens + bs - 1) // bs
    blocks = int(math.ceil(1.25 * need.sum())) + 1
    perm = rng.permutation(blocks)
    t = np.zeros((len(lens), max(1, int(need.max()))), dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        t[s, :n] = perm[at:at + n]
        at += n
    return blocks, t


def _lengths(case):
    """Per sequence: query rows, and the context after the step (decode lengths and chunk contexts are part of the
    case, not of the seed, so that the work of a case is one number)."""
    rng = np.random.default_rng(7)
    if case["op"] == "decode":
        n = case["seqs"]
        if n == 4 and case["hi"] == 300:
            return np.ones(4, dtype=np.int64), np.array([41, 129, 301, 65])
        return np.ones(n, dtype=np.int64), rng.integers(case["lo"], case["hi"] + 1, n)
    prior = rng.integers(case["prior"] // 2 if case["chunks"] < 4 else 0, case["prior"] + 1, case["chunks"])
    rows = np.full(case["chunks"], case["rows"])
    dec = rng.integers(min(64, case["hi"]), case["hi"] + 1, case["decodes"]) if case["decodes"] else np.zeros(0, dtype=np.int64)
    return np.concatenate([rows, np.ones(case["decodes"], dtype=np.int64)]), np.concatenate([prior + rows, dec])


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = _DT[case["q"]]
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    st = dict(case=case)
    if case["op"] in ("prep", "read"):
        n = case["tokens"]
        # the tokens' slots: runs of whole blocks in shuffled order, as several sequences' tokens lie in a pool; a
        # decode step's tokens (up to 256) each lie in a block of their own
        if case["op"] == "prep" and n <= 256:
            blocks = int(1.25 * n) + 2
            slots = rng.permutation(blocks)[:n] * bs + rng.integers(0, bs, n)
        else:
            need = (n + bs - 1) // bs
            blocks = int(1.25 * need) + 1
            slots = (rng.permutation(blocks)[:need, None] * bs + np.arange(bs)[None, :]).reshape(-1)[:n]
        st["slots"] = torch.from_numpy(slots.astype(np.int64)).to(DEV)
        st["k_cache"], st["v_cache"] = _pools(case, blocks, g)
    if case["op"] == "prep":
        # queries, keys and values as slices of one projection's output
        qkv = torch.randn((n, hq + 2 * hkv, d), generator=g, device=DEV, dtype=dt)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        st["q_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt)
        st["k_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt)
        st["eps"] = 1e-6
        rot = case["rot"]
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        angle = torch.arange(case["positions"], device=DEV, dtype=torch.float64)[:, None] * freq[None]
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        st["pos"] = torch.from_numpy(rng.integers(0, case["positions"], n).astype(np.int32)).to(DEV)
        st["q_out"] = torch.empty((n, hq, d), device=DEV, dtype=dt)
    elif case["op"] == "read":
        st["k_out"] = torch.empty((n, hkv, d), device=DEV, dtype=dt)
        st["v_out"] = torch.empty((n, hkv, d), device=DEV, dtype=dt)
    else:
        qlen, lens = _lengths(case)
        blocks, tables = _tables(lens, bs, rng)
        st["k_cache"], st["v_cache"] = _pools(case, blocks, g)
        rows = int(qlen.sum())
        # scores of some units' spread, as the cap and the biases meet them
        st["q"] = 3 * torch.randn((rows, hq, d), generator=g, device=DEV, dtype=dt)
        st["tables"] = torch.from_numpy(tables).to(DEV)
        st["lens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
        qsl = np.concatenate([[0], np.cumsum(qlen)])
        st["qsl"] = torch.from_numpy(qsl.astype(np.int32)).to(DEV)
        st["slopes"] = (torch.from_numpy((2.0 ** (-8.0 * (np.arange(hq) + 1) / hq)).astype(np.float32)).to(DEV)
                        if case["slopes"] else None)
        st["prefix"] = torch.from_numpy(np.minimum(case["prefix"], lens).astype(np.int32)).to(DEV) if case["prefix"] else None
        st["scale"] = 1 / math.sqrt(d)
        st["max_q"] = int(qlen.max())
        st["out"] = torch.empty((rows, hq, d), device=DEV, dtype=dt)
        # sequences by their query rows: the chunks, then the single-token rows
        n = case["chunks"] if case["op"] == "chunk" else 0
        st["groups"] = [(a, b, int((lens[a:b].max() + bs - 1) // bs), int(qlen[a])) for a, b in ((0, n), (n, len(lens)))
                        if b > a]
    if own:
        import paged_kv_cache_452_b200 as pa
        desc = pa.CacheDesc.make(st["k_cache"].shape[0], bs, hkv, hq, d, case["kv"], case["q"], K_SCALE, V_SCALE)
        st["desc"] = desc
        if case["op"] == "prep":
            st["prep"] = pa.QkPrep.make(st["q_weight"], st["k_weight"], st["eps"], st["cos_sin"], case["inter"])
        elif case["op"] != "read":
            st["mod"] = pa.ScoreMod.make(case["cap"], case["window"], st["slopes"], st["prefix"])
            st["ws"] = pa.alloc_workspace(pa.pa_biased_workspace_size(desc, len(lens), rows), DEV)
    return st


# ---- one pass --------------------------------------------------------------------

def _pool_view(case, t):
    """The pool's values as what it holds."""
    return t.view(torch.float8_e4m3fn) if case["kv"] == "e4m3" else t


def _plain_heads(x, w, st, rotate):
    """Norm over the head, weight, rotation: fp32."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w.float()
    rot = st["case"]["rot"]
    cs = st["cos_sin"][st["pos"].long()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    r = x[..., :rot]
    if st["case"]["inter"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_prep(st):
    c = st["case"]
    blk, off = st["slots"] // c["bs"], st["slots"] % c["bs"]
    st["q_out"].copy_(_plain_heads(st["q"], st["q_weight"], st, True))
    k, v = _plain_heads(st["k"], st["k_weight"], st, True), st["v"]
    if c["kv"] == "e4m3":
        k = (k / K_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v.float() / V_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        st["v_cache"][blk, :, :, off] = v
    else:
        k = k.to(st["k_cache"].dtype)
        st["v_cache"][blk, :, off] = v
    st["k_cache"][blk, :, off] = k


def _plain_read(st):
    c = st["case"]
    blk, off = st["slots"] // c["bs"], st["slots"] % c["bs"]
    if c["kv"] == "e4m3":
        k = st["k_cache"][blk, :, off].view(torch.float8_e4m3fn).float() * K_SCALE
        v = st["v_cache"][blk, :, :, off].view(torch.float8_e4m3fn).float() * V_SCALE
    else:
        k, v = st["k_cache"][blk, :, off], st["v_cache"][blk, :, off]
    st["k_out"].copy_(k)
    st["v_out"].copy_(v)


def _plain_attend(st, a, b, blocks, rows):
    """Sequences a .. b - 1, `rows` query rows each, over their tables' first `blocks` entries."""
    c = st["case"]
    hkv, d, bs = c["hkv"], c["d"], c["bs"]
    n, grp = b - a, c["hq"] // c["hkv"]
    t = st["tables"][a:b, :blocks].long()
    k, v = st["k_cache"][t], st["v_cache"][t]  # [n][blocks][hkv][bs][d]
    if c["kv"] == "e4m3":
        k = k.view(torch.float8_e4m3fn).float() * K_SCALE
        v = v.view(torch.float8_e4m3fn).float().transpose(3, 4) * V_SCALE
    keys = blocks * bs
    k = k.float().permute(0, 2, 1, 3, 4).reshape(n, hkv, keys, d)
    v = v.float().permute(0, 2, 1, 3, 4).reshape(n, hkv, keys, d)
    lens = st["lens"][a:b].long()
    first = st["qsl"][a:b].long()
    at = first[:, None] + torch.arange(rows, device=DEV)  # [n][rows]
    q = st["q"][at].float().reshape(n, rows, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, rows * grp, d)
    s = (q @ k.transpose(2, 3)).reshape(n, hkv, rows, grp, keys) * st["scale"]
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    i = (lens[:, None] - rows + torch.arange(rows, device=DEV))[:, :, None]  # [n][rows][1]
    j = torch.arange(keys, device=DEV)
    if st["slopes"] is not None:
        s = s - st["slopes"].reshape(hkv, 1, grp, 1) * (i - j).abs().float()[:, None, :, None]
    seen = j <= i
    if c["window"]:
        seen = seen & (i - j < c["window"])
    if st["prefix"] is not None:
        seen = seen | (j < st["prefix"][a:b, None, None])
    seen = (seen & (j < lens[:, None, None]))[:, None, :, None]
    s = torch.where(seen, s, float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = torch.where(seen, p, 0.0)
    o = (p.reshape(n, hkv, rows * grp, keys) @ v).reshape(n, hkv, rows, grp, d) / p.sum(-1, keepdim=True)
    st["out"][at] = o.permute(0, 2, 1, 3, 4).reshape(n, rows, c["hq"], d).to(st["out"].dtype)


def run(st):
    c = st["case"]
    if own:
        import paged_kv_cache_452_b200 as pa
    if c["op"] == "prep":
        if own:
            pa.pa_norm_rope_write(st["desc"], st["prep"], st["q"], st["k"], st["v"], st["pos"], st["slots"], st["q_out"],
                                  st["k_cache"], st["v_cache"])
        else:
            _plain_prep(st)
        return [st["q_out"], _pool_view(c, st["k_cache"]), _pool_view(c, st["v_cache"])]
    if c["op"] == "read":
        if own:
            pa.pa_cache_read(st["desc"], st["slots"], st["k_cache"], st["v_cache"], st["k_out"], st["v_out"])
        else:
            _plain_read(st)
        return [st["k_out"], st["v_out"]]
    if own and c["op"] == "decode":
        pa.pa_decode_biased(st["desc"], st["mod"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"],
                            st["scale"], st["out"], st["ws"])
    elif own:
        pa.pa_decode_chunked_prefill_biased(st["desc"], st["mod"], st["q"], st["k_cache"], st["v_cache"], st["tables"],
                                            st["qsl"], st["lens"], st["max_q"], st["scale"], st["out"], st["ws"])
    else:
        for group in st["groups"]:  # two at most: the chunks, the single-token rows
            _plain_attend(st, *group)
    return st["out"]


# ---- what a pass cannot do without -------------------------------------------------

_BYTES = {"f32": 4, "bf16": 2, "e4m3": 1}


def work(case):
    bq, bk = _BYTES[case["q"]], _BYTES[case["kv"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "prep":
        n = case["tokens"]
        # rows in, rows out, slot and position, and the rotation table's rows (no more of them than the table has)
        nbytes = n * ((2 * hq + 2 * hkv) * d * bq + 2 * hkv * d * bk + 12) + min(n, case["positions"]) * case["rot"] * 4 + 2 * d * bq
        return dict(bytes=nbytes, flops=n * (hq + hkv) * (5 * d + 3 * case["rot"]))
    if case["op"] == "read":
        return dict(bytes=case["tokens"] * (2 * hkv * d * (bq + bk) + 8), flops=case["tokens"] * 2 * hkv * d * (bk == 1))
    qlen, lens = _lengths(case)
    w = case["window"] or (1 << 40)
    pairs = keys = 0
    for r, n in zip(qlen.tolist(), lens.tolist()):
        pfx = min(case["prefix"], n)
        i = np.arange(n - r, n)
        lo = np.maximum(0, i - w + 1)
        # the window's keys and the prefix's outside it
        pairs += int((i + 1 - lo).sum() + np.minimum(pfx, lo).sum() + np.maximum(0, pfx - i - 1).sum())
        keys += n - int(lo[0]) + min(pfx, int(lo[0]))
    rows = int(qlen.sum())
    return dict(bytes=keys * 2 * hkv * d * bk + 2 * rows * hq * d * bq + keys // case["bs"] * 4, flops=4 * hq * d * pairs)


# ---- the definition in 64 bits -------------------------------------------------------

def _e4m3(x):
    """x rounded to the e4m3 grid, ties to even, saturating."""
    e = torch.frexp(x)[1].double() - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    st = prepare(case, seed)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    scale_k, scale_v = (float(np.float32(s)) if case["kv"] == "e4m3" else 1.0 for s in (K_SCALE, V_SCALE))
    k_pool, v_pool = (_pool_view(case, st[n]) for n in ("k_cache", "v_cache"))
    if case["op"] == "read":
        flat_k = k_pool.to(torch.float32).permute(0, 2, 1, 3).reshape(-1, hkv, d)
        v = v_pool.to(torch.float32)
        flat_v = (v.permute(0, 3, 1, 2) if case["kv"] == "e4m3" else v.permute(0, 2, 1, 3)).reshape(-1, hkv, d)
        return [flat_k[st["slots"]].double() * scale_k, flat_v[st["slots"]].double() * scale_v]
    if case["op"] == "prep":
        def head(x, w):
            x = x.double()
            y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + st["eps"]) * w.double()
            half = case["rot"] // 2
            first = torch.arange(half, device=DEV) * (2 if case["inter"] else 1)
            second = first + (1 if case["inter"] else half)
            turn = st["cos_sin"].double()[st["pos"].long()]
            z = torch.complex(y[..., first], y[..., second]) * torch.complex(turn[:, :half], turn[:, half:])[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            return y
        q, k, v = head(st["q"], st["q_weight"]), head(st["k"], st["k_weight"]), st["v"].double()
        if case["kv"] == "e4m3":
            k, v = _e4m3(k / scale_k), _e4m3(v / scale_v)
        pk, pv = k_pool.to(torch.float32).double(), v_pool.to(torch.float32).double()
        where = st["slots"]
        pk.permute(0, 2, 1, 3)[where // bs, where % bs] = k
        (pv.permute(0, 3, 1, 2) if case["kv"] == "e4m3" else pv.permute(0, 2, 1, 3))[where // bs, where % bs] = v
        return [q, pk, pv]
    out = torch.zeros((st["q"].shape[0], hq, d), device=DEV, dtype=torch.float64)
    qsl, lens = st["qsl"].tolist(), st["lens"].tolist()
    for s, n in enumerate(lens):
        t = st["tables"][s, :(n + bs - 1) // bs].long()
        k = k_pool[t].to(torch.float32).double().transpose(0, 1).reshape(hkv, -1, d)[:, :n] * scale_k
        v = v_pool[t].to(torch.float32).double() * scale_v
        v = (v.transpose(2, 3) if case["kv"] == "e4m3" else v).transpose(0, 1).reshape(hkv, -1, d)[:, :n]
        r0, r1 = qsl[s], qsl[s + 1]
        dist = torch.arange(n - (r1 - r0), n, device=DEV)[:, None] - torch.arange(n, device=DEV)[None]
        hidden = dist < 0
        if case["window"]:
            hidden |= dist >= case["window"]
        if case["prefix"]:
            hidden[:, :min(case["prefix"], n)] = False
        for h in range(hq):
            x = st["q"][r0:r1, h].double() @ k[h * hkv // hq].T / math.sqrt(d)
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case["slopes"]:
                x = x - float(st["slopes"][h]) * dist.abs()
            out[r0:r1, h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v[h * hkv // hq]
    return out
