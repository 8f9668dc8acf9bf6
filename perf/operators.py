"""The operators of a sparse-attention layer around the indexer, as cases to measure.

What a layer runs beside the indexer's own scoring and selection: the norm that makes its FP8 input
rows (root mean square, with the residual's addition), the paged append of the latent and its rotated
key part, the attention of every query over the positions that the indexer selected for it, and the
attention of a batch over a prefix that all its sequences share.

``run`` computes each operator in plain torch operations, or with the library's calls where ``own`` is
set; ``exact`` is the definition in 64 bits.
"""

import math

import torch

own = False

D_C, D_R = 512, 64                     # latent values per token (the value and most of the key), rotated key part
SM_SCALE = 1.0 / math.sqrt(192.0)      # heads of 128 + 64 values before the latent projection is absorbed
E4M3_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # a decode step's rows: latency, one 7168-wide hidden row per sequence, FP8 groups of 128 for the projections
        dict(name="norm step", op="norm", rows=4, d=7168, dtype="bf16", residual=True, group=128, pad=0),
        # a long prompt's rows: bandwidth
        dict(name="norm prompt", op="norm", rows=16384, d=7168, dtype="bf16", residual=True, group=128, pad=0),
        # a low-rank slice of a wider fp32 projection, one scale per row, an odd row count
        dict(name="norm slice", op="norm", rows=1023, d=1536, dtype="f32", residual=False, group=0, pad=576),
        # one decode step of 32 sequences into a bf16 cache
        dict(name="append step", op="append", n=32, seqs=32, page=64, fp8=False, interleaved=True, far=32768),
        # a prompt chunk into an FP8 cache, pages of 64
        dict(name="append prompt", op="append", n=16384, seqs=3, page=64, fp8=True, interleaved=True, far=0),
        # a single query over the selection of a long sequence: latency, the selection split over the GPU
        dict(name="select one", op="select", T=1, H=128, k=2048, length=32768, per_seq=True, fp8=False, page=64, hole=0.0),
        # a decode batch, every query with its own sequence
        dict(name="select batch", op="select", T=64, H=128, k=2048, length=16384, per_seq=True, fp8=False, page=64, hole=0.0),
        # one of eight ranks' heads, an FP8 cache, short selections padded with -1
        dict(name="select few heads", op="select", T=37, H=16, k=2048, length=9001, per_seq=True, fp8=True, page=16, hole=0.3),
        # the end of a long prompt: many queries of one sequence
        dict(name="select prompt", op="select", T=1024, H=128, k=2048, length=16384, per_seq=False, fp8=False, page=64, hole=0.0),
        # two sequences behind a short shared system prompt
        dict(name="prefix short", op="prefix", T=2, H=128, prefix=500, suffix=100, fp8=False, page=64),
        # a serving batch behind one long document, one of eight ranks' heads
        dict(name="prefix batch", op="prefix", T=64, H=16, prefix=32768, suffix=1024, fp8=False, page=64),
        # all heads, an FP8 cache, an odd batch and a prefix that ends inside a page
        dict(name="prefix wide", op="prefix", T=23, H=128, prefix=16001, suffix=777, fp8=True, page=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "select", "select", "prefix", "prefix"])
    if op == "norm":
        d = 16 * _log(rng, 8, 448)
        return dict(op=op, rows=_log(rng, 1, 16384), d=d, dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.6,
                    group=rng.choice([0, 128]), pad=16 * rng.choice([0, 0, 4, 33]))
    if op == "append":
        return dict(op=op, n=_log(rng, 1, 16384), seqs=rng.randint(1, 40), page=rng.choice([1, 16, 48, 64, 256]), fp8=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, far=rng.choice([0, 0, 100000]))
    H = rng.choice([8, 16, 24, 32, 64, 96, 128, 128])
    if op == "select":
        k = rng.choice([2048, 2048, _log(rng, 1, 2048)])
        return dict(op=op, T=_log(rng, 1, 200), H=H, k=k, length=k + _log(rng, 1, 16384), per_seq=rng.random() < 0.7,
                    fp8=rng.random() < 0.4, page=rng.choice([16, 48, 64, 256]), hole=rng.choice([0.0, 0.0, 0.5]))
    return dict(op=op, T=_log(rng, 1, 64), H=H, prefix=rng.choice([0, _log(rng, 1, 16384), _log(rng, 64, 16384)]), suffix=_log(rng, 1, 2048),
                fp8=rng.random() < 0.4, page=rng.choice([16, 48, 64, 256]))


# ------------------------------------------------------------------------------------------------ inputs


def _torch_dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _pow2_scale(amax):
    """The smallest power of two that brings amax to at most 448 (1 for a row of zeros)."""
    e = torch.ceil(torch.log2((amax / E4M3_MAX).clamp_min(2.0 ** -100)))
    e = torch.where(torch.exp2(e) * E4M3_MAX < amax, e + 1, e)
    e = torch.where(torch.exp2(e - 1) * E4M3_MAX >= amax, e - 1, e)
    return torch.where(amax > 0, torch.exp2(e), torch.ones_like(amax))


def _cache(rows, fp8, g):
    """A latent cache with contents: latent, scale (None in bf16), rotated key part."""
    latent = torch.empty(rows, D_C, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    scale = torch.empty(rows, dtype=torch.float32, device="cuda") if fp8 else None
    for r in range(0, rows, 1 << 18):
        x = torch.randn(min(1 << 18, rows - r), D_C, dtype=torch.float32, device="cuda", generator=g)
        if fp8:
            s = _pow2_scale(x.abs().amax(1))
            scale[r:r + len(x)] = s
            latent[r:r + len(x)] = (x / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            latent[r:r + len(x)] = x.to(torch.bfloat16)
    rope = torch.randn(rows, D_R, dtype=torch.float32, device="cuda", generator=g).to(torch.bfloat16)
    return latent, scale, rope


def _table(seqs, pages, shared, g):
    """Page tables of `seqs` sequences of `pages` pages each, in no order, the first `shared` pages the same for all."""
    total = shared + seqs * (pages - shared)
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    own_pages = perm[shared:].view(seqs, pages - shared)
    return torch.cat([perm[:shared].expand(seqs, shared), own_pages], 1).contiguous(), total


def _lib_cache(st):
    from sparse_attention_token_02_b200 import api
    return api.LatentCache(st["latent"], st["rope"], st["scale"], st["page"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    if case["op"] == "norm":
        dt, rows, d = _torch_dtype(case["dtype"]), case["rows"], case["d"]
        wide = torch.randn(rows, d + case["pad"], dtype=torch.float32, device="cuda", generator=g).to(dt)
        st["x"] = wide[:, :d]
        st["residual"] = (3 * torch.randn(rows, d, dtype=torch.float32, device="cuda", generator=g)).to(dt) if case["residual"] else None
        st["weight"] = (1 + 0.1 * torch.randn(d, dtype=torch.float32, device="cuda", generator=g)).to(torch.bfloat16)
        return st
    if case["op"] == "append":
        n, seqs, page = case["n"], case["seqs"], case["page"]
        seq = torch.arange(n, device="cuda") * seqs // n if n >= seqs else torch.randperm(seqs, device="cuda", generator=g)[:n].sort().values
        first = torch.searchsorted(seq, seq)                           # the first token of each token's sequence
        pos = torch.arange(n, device="cuda") - first
        pages = -(-(n + 64) // page)
        if case["far"]:                                                # a long history: only its last pages are resident here
            start = torch.randint(case["far"] // 2, case["far"], (seqs,), device="cuda", generator=g)
            pos = pos + start[seq]
            pages = -(-(case["far"] + n) // page)
        live = torch.zeros(seqs, pages, dtype=torch.bool, device="cuda")
        live[seq, pos // page] = True
        count = int(live.sum())
        table = torch.full((seqs, pages), -1, dtype=torch.int32, device="cuda")
        table[live] = torch.randperm(count, device="cuda", generator=g).to(torch.int32)
        rows = count * page
        st["latent"] = torch.zeros(rows, D_C, dtype=torch.uint8 if case["fp8"] else torch.bfloat16, device="cuda")
        st["scale"] = torch.ones(rows, dtype=torch.float32, device="cuda") if case["fp8"] else None
        st["rope"] = torch.zeros(rows, D_R, dtype=torch.bfloat16, device="cuda")
        both = torch.randn(n, D_C + D_R, dtype=torch.float32, device="cuda", generator=g).to(torch.bfloat16)   # one projection's output
        st.update(c_new=both[:, :D_C], kr_new=both[:, D_C:], table=table, seq_ids=seq.to(torch.int32), positions=pos.to(torch.int32))
        return st
    T, H, page = case["T"], case["H"], case["page"]
    st["q_latent"] = torch.randn(T, H, D_C, dtype=torch.float32, device="cuda", generator=g).to(torch.bfloat16)
    st["q_rope"] = torch.randn(T, H, D_R, dtype=torch.float32, device="cuda", generator=g).to(torch.bfloat16)
    if case["op"] == "select":
        k, length = case["k"], case["length"]
        seqs = T if case["per_seq"] else 1
        st["table"], total = _table(seqs, -(-length // page), 0, g)
        st["seq_ids"] = torch.arange(T, dtype=torch.int32, device="cuda") if case["per_seq"] else torch.zeros(T, dtype=torch.int32, device="cuda")
        idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
        for t0 in range(0, T, 64):                                    # k distinct positions a query, in no order
            m = min(64, T - t0)
            idx[t0:t0 + m] = torch.rand(m, length, device="cuda", generator=g).topk(k, 1).indices.to(torch.int32)
        if case["hole"]:                                              # valid entries first, then padding
            keep = (torch.rand(T, device="cuda", generator=g) * case["hole"] * 2 * k).to(torch.int64)
            idx.masked_fill_(torch.arange(k, device="cuda")[None, :] >= (k - keep).clamp_min(1)[:, None], -1)
        st["idx"] = idx
    else:
        prefix, suffix = case["prefix"], case["suffix"]
        lens = torch.randint(1, suffix + 1, (T,), device="cuda", generator=g)
        lens[0] = suffix
        shared = prefix // page
        st["table"], total = _table(T, -(-(prefix + suffix) // page), shared, g)
        st["seq_ids"] = torch.arange(T, dtype=torch.int32, device="cuda")
        st["key_lens"] = (prefix + lens).to(torch.int32)
    st["latent"], st["scale"], st["rope"] = _cache(total * page, case["fp8"], g)
    if case["op"] == "prefix" and prefix % page:                       # a page that the prefix ends in: each sequence has its own copy
        rows = st["table"][:, shared].long()[:, None] * page + torch.arange(prefix % page, device="cuda")
        for t in (st["latent"], st["rope"]) + ((st["scale"],) if case["fp8"] else ()):
            t[rows] = t[rows[:1]].clone()
    return st


# ------------------------------------------------------------------------------------------------ one pass


def run(st):
    return {"norm": _run_norm, "append": _run_append, "select": _run_select, "prefix": _run_prefix}[st["op"]](st)


def _run_norm(st):
    x, res, w, group = st["x"], st["residual"], st["weight"], st["group"]
    if own:
        from sparse_attention_token_02_b200 import api
        out = api.dsa_rmsnorm_fp8(x, w, EPS, residual=res, group=group)
        return {"codes": out[0].view(torch.float8_e4m3fn), "scale": out[1], "residual": out[2]}
    s = x.float() if res is None else x.float() + res.float()
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * w.float()
    rows, d = y.shape
    step = group or d
    n = -(-d // step)
    y = torch.nn.functional.pad(y, (0, n * step - d)).view(rows, n, step)
    amax = y.abs().amax(2)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    codes = (y / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    codes = codes.view(torch.uint8).view(rows, n * step)[:, :d].contiguous().view(torch.float8_e4m3fn)
    return {"codes": codes, "scale": scale, "residual": None if res is None else s.to(x.dtype)}


def _run_append(st):
    if own:
        from sparse_attention_token_02_b200 import api
        api.dsa_latent_append_rope(_lib_cache(st), st["table"], st["c_new"], st["kr_new"], st["seq_ids"], st["positions"],
                                   interleaved=st["interleaved"])
    else:
        pos = st["positions"].long()
        page = st["page"]
        row = st["table"][st["seq_ids"].long(), pos // page].long() * page + pos % page
        theta = pos[:, None].double() * 10000.0 ** (-torch.arange(0, D_R, 2, device="cuda", dtype=torch.float64) / D_R)
        c, s = torch.cos(theta).float(), torch.sin(theta).float()
        kr = st["kr_new"].float()
        a, b = (kr[:, 0::2], kr[:, 1::2]) if st["interleaved"] else (kr[:, :D_R // 2], kr[:, D_R // 2:])
        u, v = a * c - b * s, a * s + b * c
        st["rope"][row] = (torch.stack([u, v], 2).flatten(1) if st["interleaved"] else torch.cat([u, v], 1)).to(torch.bfloat16)
        x = st["c_new"].float()
        if st["fp8"]:
            scale = _pow2_scale(x.abs().amax(1))
            st["scale"][row] = scale
            st["latent"][row] = (x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            st["latent"][row] = x.to(torch.bfloat16)
    if st["fp8"]:
        return {"latent": st["latent"].view(torch.float8_e4m3fn), "scale": st["scale"], "rope": st["rope"]}
    return {"latent": st["latent"], "rope": st["rope"]}


def _values(st, rows):
    """Latents and rotated parts of cache rows, in 32 bits."""
    c = st["latent"][rows]
    c = c.view(torch.float8_e4m3fn).float() * st["scale"][rows][..., None] if st["fp8"] else c.float()
    return c, st["rope"][rows].float()


def _run_select(st):
    if own:
        from sparse_attention_token_02_b200 import api
        out, lse = api.dsa_sparse_attention(st["q_latent"], st["q_rope"], _lib_cache(st), st["table"], st["seq_ids"], st["idx"], SM_SCALE)
        return {"out": out, "lse": lse}
    idx, page = st["idx"].long(), st["page"]
    at = idx.clamp_min(0)
    rows = st["table"].long()[st["seq_ids"].long()[:, None], at // page] * page + at % page
    c, r = _values(st, rows)
    s = (st["q_latent"].float() @ c.transpose(1, 2) + st["q_rope"].float() @ r.transpose(1, 2)) * SM_SCALE
    s = s.masked_fill((idx < 0)[:, None, :], -math.inf)
    m = s.amax(2, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(2, keepdim=True)
    return {"out": ((p @ c) / total).to(torch.bfloat16), "lse": (m + torch.log(total))[:, :, 0]}


def _run_prefix(st):
    if own:
        from sparse_attention_token_02_b200 import api
        out, lse = api.dsa_prefix_attention(st["q_latent"], st["q_rope"], _lib_cache(st), st["table"], st["seq_ids"], st["key_lens"], SM_SCALE,
                                            prefix_len=st["prefix"], max_keys=st["prefix"] + st["suffix"])
        return {"out": out, "lse": lse}
    T, H, page, prefix, suffix = st["T"], st["H"], st["page"], st["prefix"], st["suffix"]
    q, qr = st["q_latent"].float(), st["q_rope"].float()
    table = st["table"].long()
    at = torch.arange(prefix, device="cuda")
    c0, r0 = _values(st, table[0, at // page] * page + at % page)
    own_at = prefix + torch.arange(suffix, device="cuda")
    c1, r1 = _values(st, table[st["seq_ids"].long()][:, own_at // page] * page + own_at % page)
    s0 = (q.view(T * H, D_C) @ c0.t() + qr.view(T * H, D_R) @ r0.t()).view(T, H, prefix) * SM_SCALE
    s1 = (q @ c1.transpose(1, 2) + qr @ r1.transpose(1, 2)) * SM_SCALE
    s1 = s1.masked_fill((own_at[None, :] >= st["key_lens"][:, None])[:, None, :], -math.inf)
    s = torch.cat([s0, s1], 2)
    m = s.amax(2, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(2, keepdim=True)
    o = (p[:, :, :prefix].reshape(T * H, prefix) @ c0).view(T, H, D_C) + p[:, :, prefix:] @ c1
    return {"out": (o / total).to(torch.bfloat16), "lse": (m + torch.log(total))[:, :, 0]}


# ------------------------------------------------------------------------------------------------ the least work


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["d"]
        e = 2 if case["dtype"] == "bf16" else 4
        groups = case["rows"] * (-(-case["d"] // case["group"]) if case["group"] else 1)
        return {"bytes": n * (e + 1) + (2 * n * e if case["residual"] else 0) + 2 * case["d"] + 4 * groups, "flops": 8 * n}
    if case["op"] == "append":
        n = case["n"]
        return {"bytes": n * (2 * (D_C + D_R) + (D_C + 4 if case["fp8"] else 2 * D_C) + 2 * D_R + 12), "flops": n * (2 * D_C + 6 * D_R)}
    T, H = case["T"], case["H"]
    row = (D_C + 4 if case["fp8"] else 2 * D_C) + 2 * D_R
    ends = T * H * (2 * (D_C + D_R) + 2 * D_C + 4)                      # queries, outputs, logs of sums
    if case["op"] == "select":
        valid = T * case["k"] * (1 - case["hole"])                     # the mean of the drawn paddings
        keys = valid if case["per_seq"] else min(valid, case["length"])
        return {"bytes": int(keys * row + T * case["k"] * 4 + ends), "flops": int(2 * valid * H * (2 * D_C + D_R))}
    keys = T * (case["prefix"] + (case["suffix"] + 1) / 2)
    return {"bytes": int((case["prefix"] + T * (case["suffix"] + 1) / 2) * row + ends), "flops": int(2 * keys * H * (2 * D_C + D_R))}


# ------------------------------------------------------------------------------------------------ 64 bits


def _e4m3_nearest(v):
    """The E4M3 values nearest to v (64 bits), ties to the even code, saturated at 448."""
    a = v.abs().clamp_max(E4M3_MAX)
    _, e = torch.frexp(a)                                               # a = m * 2^e, m in [0.5, 1)
    step = torch.exp2((e.double() - 4).clamp_min(-9))                   # three mantissa bits, subnormal steps of 2^-9
    return torch.copysign(torch.round(a / step) * step, v)


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "select": _exact_select, "prefix": _exact_prefix}[case["op"]](st)


def _exact_norm(st):
    d, group = st["d"], st["group"] or st["d"]
    codes, scales, sums = [], [], []
    for r in range(0, st["rows"], 2048):
        s = st["x"][r:r + 2048].double()
        if st["residual"] is not None:
            s = s + st["residual"][r:r + 2048].double()
            sums.append(s)
        y = s / torch.sqrt(s.square().sum(1, keepdim=True) / d + EPS) * st["weight"].double()
        parts = [y[:, i:i + group] for i in range(0, d, group)]
        sc = [p.abs().max(1).values / E4M3_MAX for p in parts]
        sc = [torch.where(v == 0, torch.ones_like(v), v) for v in sc]
        codes.append(torch.cat([_e4m3_nearest(p / v[:, None]) for p, v in zip(parts, sc)], 1))
        scales.append(torch.stack(sc, 1))
    return {"codes": torch.cat(codes), "scale": torch.cat(scales), "residual": torch.cat(sums) if sums else None}


def _exact_append(st):
    rows = st["latent"].shape[0]
    latent = torch.zeros(rows, D_C, dtype=torch.float64, device="cuda")
    rope = torch.zeros(rows, D_R, dtype=torch.float64, device="cuda")
    scale = torch.ones(rows, dtype=torch.float64, device="cuda")
    pos, seq = st["positions"].long(), st["seq_ids"].long()
    page_of = st["table"].long()[seq, torch.div(pos, st["page"], rounding_mode="floor")]
    at = page_of * st["page"] + torch.remainder(pos, st["page"])
    x = st["c_new"].double()
    if st["fp8"]:
        amax = x.abs().max(1).values
        m, e = torch.frexp(amax / E4M3_MAX)                             # amax / 448 = m * 2^e: a power of two where m is 1/2
        s = torch.where(amax == 0, torch.ones_like(amax), torch.exp2(torch.where(m == 0.5, e - 1, e).double()))
        scale[at], latent[at] = s, _e4m3_nearest(x / s[:, None])
    else:
        latent[at] = x
    z = st["kr_new"].double()
    half = D_R // 2
    z = torch.complex(z[:, 0::2].contiguous(), z[:, 1::2].contiguous()) if st["interleaved"] else torch.complex(z[:, :half].contiguous(), z[:, half:].contiguous())
    freq = torch.exp(-math.log(10000.0) * torch.arange(half, device="cuda", dtype=torch.float64) / half)
    z = z * torch.polar(torch.ones_like(pos, dtype=torch.float64)[:, None].expand(-1, half).contiguous(), pos.double()[:, None] * freq)
    rope[at] = torch.view_as_real(z).flatten(1) if st["interleaved"] else torch.cat([z.real, z.imag], 1)
    return {"latent": latent, "scale": scale, "rope": rope} if st["fp8"] else {"latent": latent, "rope": rope}


def _exact_rows(st, rows):
    c = st["latent"].index_select(0, rows)
    if st["fp8"]:
        c = c.view(torch.float8_e4m3fn).double() * st["scale"].index_select(0, rows).double().unsqueeze(1)
    return torch.cat([c.double(), st["rope"].index_select(0, rows).double()], 1)


def _exact_attend(q, keys):
    s = q @ keys.t() * SM_SCALE
    lse = torch.logsumexp(s, 1)
    return torch.exp(s - lse[:, None]) @ keys[:, :D_C], lse


def _exact_select(st):
    outs = []
    q = torch.cat([st["q_latent"], st["q_rope"]], 2).double()
    for t in range(st["T"]):
        pos = st["idx"][t].long()
        pos = pos[pos >= 0]
        table = st["table"][int(st["seq_ids"][t])].long()
        outs.append(_exact_attend(q[t], _exact_rows(st, table[pos // st["page"]] * st["page"] + pos % st["page"])))
    return {"out": torch.stack([o for o, _ in outs]), "lse": torch.stack([x for _, x in outs])}


def _exact_prefix(st):
    outs = []
    q = torch.cat([st["q_latent"], st["q_rope"]], 2).double()
    for t in range(st["T"]):
        pos = torch.arange(int(st["key_lens"][t]), device="cuda")
        table = st["table"][t].long()
        outs.append(_exact_attend(q[t], _exact_rows(st, table[pos // st["page"]] * st["page"] + pos % st["page"])))
    return {"out": torch.stack([o for o, _ in outs]), "lse": torch.stack([x for _, x in outs])}
