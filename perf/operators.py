"""Cases that measure the cache-side operators of an attention layer: appending
rotated keys (and rotating the queries) into the striped paged pool, attention
over a pool held in 4 bits, and attention whose scores are capped by a tanh or
lowered linearly with the distance.

``own`` False computes each operator in its plain form (elementary torch
operations in 32 bits, rounded once at the end); ``own`` True makes the calls a
user makes of the library.  ``exact`` gives the same results in 64 bits, laid
out by another route than the plain form's.

A case is a dict of plain values:

  op      "append" (rotation + append) or "attend" (a step's attention)
  pool    bf16, fp32, e4m3 or fp4: type of the pool's rows (fp32: an fp32 layer)
  rows    requests of the step; row i brings between new_lo and new_hi new
          tokens after between ctx_lo and ctx_hi cached ones (evenly spread,
          shuffled by the seed); pad: tokens of no row at the end
  hq, hkv, d, p, page, il   heads, head width, partners, page size, interleave
  style, rot, rot_begin     rotation: pairing, width, first rotated value
  cap, slopes, q_std        score cap (0: none), distance slopes, spread of the queries
  append  an "attend" step that first rotates and appends its new tokens
"""

import math

import torch

own = False

_MLA_D, _MLA_DV = 576, 512
_DESCALE = {"bf16": (1.0, 1.0), "fp32": (1.0, 1.0), "e4m3": (0.0123, 0.0137), "fp4": (0.0021, 0.0023)}


def _case(name, op, pool, rows, new, ctx, hq, hkv, d, p, page, il=1, style="halves", rot=0, rot_begin=0, cap=0.0,
          slopes=False, q_std=1.0, append=False, pad=0):
    c = {"op": op, "pool": pool, "rows": rows, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0],
         "ctx_hi": ctx[1], "hq": hq, "hkv": hkv, "d": d, "p": p, "page": page, "il": il, "style": style,
         "rot": rot, "rot_begin": rot_begin, "cap": cap, "slopes": slopes, "q_std": q_std, "append": append,
         "pad": pad}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's append: 64 requests, one token each, before the attention call
        _case("append decode bf16", "append", "bf16", 64, (1, 1), (511, 8191), 32, 8, 128, 4, 16, rot=128),
        # a prompt batch of uneven lengths going into an E4M3 pool, half of every head rotated
        _case("append prompt e4m3", "append", "e4m3", 16, (2, 1021), (0, 4000), 64, 8, 128, 8, 64, style="pairs",
              rot=64),
        # latent rows of a prompt: the last 64 of 576 values rotate, and 128 query heads with them
        _case("append latent bf16", "append", "bf16", 5, (1, 407), (0, 9000), 128, 1, _MLA_D, 4, 64, style="pairs",
              rot=64, rot_begin=512),
        # two requests of a small fp32 layer (interactive use: latency)
        _case("append tiny fp32", "append", "fp32", 2, (1, 1), (36, 99), 4, 1, 64, 2, 16, il=4, rot=32, pad=1),
        # the decode batch of the headline benchmark over a 4-bit pool
        _case("fp4 decode", "attend", "fp4", 64, (1, 1), (511, 8191), 32, 8, 128, 4, 16),
        # a few short requests, append and attention as one step (latency)
        _case("fp4 append+decode short", "attend", "fp4", 3, (1, 1), (0, 700), 32, 8, 128, 4, 16, il=2, rot=128,
              append=True),
        # long contexts over a 4-bit pool: what 4 bits are for
        _case("fp4 decode long", "attend", "fp4", 8, (1, 1), (65535, 131071), 64, 8, 128, 8, 64),
        # prompt pieces over cached 4-bit context, their own tokens in bf16
        _case("fp4 prompt pieces", "attend", "fp4", 16, (2, 256), (0, 8192), 32, 8, 128, 4, 16, pad=7),
        # the decode batch with capped scores
        _case("capped decode bf16", "attend", "bf16", 64, (1, 1), (511, 8191), 32, 8, 128, 4, 16, cap=30.0,
              q_std=8.0),
        # long E4M3 contexts with a slope for each head
        _case("slopes decode e4m3", "attend", "e4m3", 8, (1, 1), (16384, 65535), 64, 8, 128, 8, 64, slopes=True),
        # prompt pieces with both, their own tokens too
        _case("capped+slopes pieces", "attend", "bf16", 16, (2, 256), (0, 8192), 32, 8, 128, 4, 16, cap=50.0,
              slopes=True, q_std=8.0),
        # two short fp32 rows (latency)
        _case("capped tiny fp32", "attend", "fp32", 2, (1, 1), (36, 99), 4, 1, 64, 2, 16, cap=20.0, slopes=True,
              q_std=4.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    p = rng.choice([1, 2, 4, 8])
    il = rng.choice([1, 1, 2, 4])
    page = p * il * rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    if rng.random() < 0.4:
        pool = rng.choice(["bf16", "e4m3", "fp32"])
        g = rng.choice([1, 2, 4, 8, 16])
        rows = _log(rng, 1, 24)
        hi = _log(rng, 1, max(2, min(900, int(1e8 / (rows * hkv * g * d)))))
        ctx = _log(rng, 1, 20000)
        rot = 2 * rng.randint(4, d // 2)
        return _case("", "append", pool, rows, (rng.randint(1, hi), hi), (rng.randint(0, ctx), ctx),
                     hkv * g, hkv, d, p, page, il=il, style=rng.choice(["halves", "pairs"]), rot=rot,
                     rot_begin=rng.choice([0, d - rot]), pad=rng.randint(0, 9))
    pool = rng.choice(["fp4", "fp4", "bf16", "e4m3", "fp32"])
    mod = pool != "fp4" or rng.random() < 0.3
    cap = round(rng.uniform(10.0, 60.0), 1) if mod and rng.random() < 0.7 else 0.0
    slopes = mod and (cap == 0.0 or rng.random() < 0.5)
    g = rng.choice([1, 2, 4, 8] if pool == "fp32" else [1, 2, 4, 8, 16])
    append = rng.random() < 0.3
    if rng.random() < 0.6:  # one token a row
        rows = _log(rng, 1, 64)
        ctx = _log(rng, 1, min(100000, (100000 if pool == "fp32" else 250000) // rows))
        new = (1, 1)
    else:
        rows = _log(rng, 1, 12)
        ctx = _log(rng, 1, 8000)
        hi = _log(rng, 2, max(3, min(200, int(6e8 / (rows * ctx * hkv * g)))))
        new = (1, hi)
    return _case("", "attend", pool, rows, new, (rng.randint(0, ctx), ctx), hkv * g, hkv, d, p, page, il=il,
                 rot=d if append else 0, cap=cap, slopes=slopes, q_std=round(rng.uniform(0.5, 8.0), 2),
                 append=append, pad=rng.randint(0, 5))


# ---- sizes that follow from a case alone

def _spread(n, lo, hi):
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(c):
    """(new tokens, cached tokens) of each row, before the shuffle."""
    return _spread(c["rows"], c["new_lo"], c["new_hi"]), _spread(c["rows"], c["ctx_lo"], c["ctx_hi"])[::-1]


def _decode(c):
    return c["new_lo"] == c["new_hi"] == 1


def _esz(c):
    return 4 if c["pool"] == "fp32" else 2


def _row_bytes(c, d):
    return {"bf16": 2 * d, "fp32": 4 * d, "e4m3": d, "fp4": d // 2 + d // 16}[c["pool"]]


def work(c):
    new, ctx = _lengths(c)
    t, e, d = sum(new), _esz(c), c["d"]
    mla = d == _MLA_D
    nbytes = flops = 0.0
    if c["op"] == "append" or c["append"]:
        # queries in and out, new keys in and out (k_out), values in, pool rows out, cos and sin, positions
        nbytes += t * (2 * c["hq"] * d * e + 2 * c["hkv"] * d * e + (0 if mla else c["hkv"] * d * e))
        nbytes += t * (c["hkv"] * _row_bytes(c, d) * (1 if mla else 2) + c["rot"] * 4 + 4)
        flops += t * (c["hq"] + c["hkv"]) * c["rot"] * 3
    if c["op"] == "attend":
        keys = sum(ctx) + (t if _decode(c) else 0)
        pairs = sum(n * m for n, m in zip(new, ctx)) + sum(n * (n + 1) // 2 for n in new)
        nbytes += keys * c["hkv"] * 2 * _row_bytes(c, d) + t * c["hq"] * (2 * d * e + 4)
        nbytes += 0 if _decode(c) else t * c["hkv"] * 2 * d * e
        flops += 4.0 * pairs * c["hq"] * d
    return {"bytes": nbytes, "flops": flops}


# ---- 4-bit rows: codes of magnitude 0 0.5 1 1.5 2 3 4 6 (bit 3 the sign, even
# value in the low half of a byte), a scale in E4M3 for each 16 values, and one
# descale a tensor.  A pool is one byte buffer: every row's codes, then every
# row's scales.

def _e4m3_bytes(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _fp4_rows(x, descale):
    """Codes [..., d / 2] and scales [..., d / 16] of rows x (32 bits)."""
    v = (x / descale).unflatten(-1, (-1, 16))
    sf = _e4m3_bytes(v.abs().amax(-1) / 6.0)
    s = sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    a = torch.where(s > 0, v.abs() / s, torch.zeros_like(v))
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * ((v < 0) & (s > 0)).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], sf


def _pool_rows(c, n_pages):
    return c["p"] * n_pages * c["hkv"] * (c["page"] // c["p"])


def _make_pool(c, n_pages, descale, gen, d):
    rows = _pool_rows(c, n_pages)
    x = torch.randn(rows, d, generator=gen, device="cuda")
    if c["pool"] == "fp4":
        codes, sf = _fp4_rows(x, descale)
        return torch.cat([codes.flatten(), sf.flatten()])
    if c["pool"] == "e4m3":
        return _e4m3_bytes(x / descale).view(c["p"], n_pages, c["hkv"], c["page"] // c["p"], d)
    return x.to(torch.float32 if c["pool"] == "fp32" else torch.bfloat16).view(
        c["p"], n_pages, c["hkv"], c["page"] // c["p"], d)


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    d, mla = c["d"], c["d"] == _MLA_D
    layer = torch.float32 if c["pool"] == "fp32" else torch.bfloat16
    new, ctx = _lengths(c)
    order = torch.randperm(c["rows"], generator=host)
    new, ctx = torch.tensor(new)[order], torch.tensor(ctx)[order]
    need = (new + ctx + c["page"] - 1) // c["page"]
    n_pages = int(need.sum()) + int(need.sum()) // 20 + 1
    indices = torch.randperm(n_pages - 1, generator=host)[: int(need.sum())]
    zero = torch.zeros(1, dtype=torch.long)
    indptr = torch.cat([zero, need.cumsum(0)])
    qo = torch.cat([zero, new.cumsum(0)])
    used = int(qo[-1])
    t = used + c["pad"]
    row = torch.repeat_interleave(torch.arange(c["rows"]), new)
    pos = torch.full((t,), -1, dtype=torch.long)
    pos[:used] = ctx[row] + torch.arange(used) - qo[row]
    kd, vd = _DESCALE[c["pool"]]
    i32 = lambda x: x.to(torch.int32).cuda()  # noqa: E731
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    mag, byte = torch.cat([mag, -mag]), torch.arange(256)
    s = {"case": c, "pairs": torch.stack([mag[byte & 15], mag[byte >> 4]], 1).cuda(),  # the values of a byte of codes
         "n_pages": n_pages, "kd": kd, "vd": vd, "scale": 1.0 / math.sqrt(192.0 if mla else d),
         "positions": i32(pos), "qo": i32(qo), "indptr": i32(indptr), "indices": i32(indices),
         "kv_len": i32(ctx + new if _decode(c) else ctx), "max_new": int(new.max()),
         "max_kv": max(1, int((ctx + new if _decode(c) else ctx).max())),
         # longest rows first, as a scheduler that knows the lengths hands them over
         "order": i32(torch.argsort(-(ctx + new), stable=True)) if _decode(c) and not c["pad"] else None,
         "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    s["pool_k"] = _make_pool(c, n_pages, kd, gen, d)
    s["pool_v"] = None if mla else _make_pool(c, n_pages, vd, gen, d)
    s["q"] = (torch.randn(t, c["hq"], d, generator=gen, device="cuda") * c["q_std"]).to(layer)
    s["k_new"] = torch.randn(t, c["hkv"], d, generator=gen, device="cuda").to(layer)
    s["v_new"] = None if mla else torch.randn(t, c["hkv"], d, generator=gen, device="cuda").to(layer)
    if c["rot"]:
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
        ang = torch.arange(int((ctx + new).max()), dtype=torch.float64)[:, None].cuda() * inv.cuda()
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["q_rot"], s["k_rot"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k_new"])
    s["slopes"] = None
    if c["slopes"]:
        s["slopes"] = (2.0 ** (-8.0 * (torch.arange(c["hq"], dtype=torch.float64) + 1) / c["hq"])).float().cuda()
    if own:
        _prepare_own(s)
    return s


# ---- the framework's calls

def _prepare_own(s):
    """What a user's program keeps between steps: the pool's description, output buffers and the workspace."""
    from context_paged_attention_gb300 import binding as B

    c = s["case"]
    kv = {"bf16": 0, "fp32": 0, "e4m3": B.DTYPE_FP8_E4M3, "fp4": B.DTYPE_FP4_E2M1}[c["pool"]]
    s["desc"] = B.PoolDesc(P=c["p"], page_size=c["page"], num_pages=s["n_pages"], num_kv_heads=c["hkv"],
                           head_dim=c["d"], head_dim_v=_MLA_DV if c["d"] == _MLA_D else c["d"],
                           dtype=B.DTYPE_FP32 if c["pool"] == "fp32" else B.DTYPE_BF16, interleave=c["il"],
                           kv_dtype=kv, k_descale=s["kd"] if kv else 0.0, v_descale=s["vd"] if kv else 0.0)
    if c["op"] == "attend":
        t = s["q"].shape[0]
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(t, c["hq"], device="cuda")
        if not _decode(c):
            s["o_own"] = torch.empty(t, c["hq"], c["d"], device="cuda")
            s["lse_own"] = torch.empty(t, c["hq"], device="cuda")
        n = B.fused_workspace_bytes(s["desc"], c["hq"], t, s["max_kv"])
        s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        s["mod"] = None
        if c["cap"] or c["slopes"]:
            s["mod"] = B.score_mod(softcap=c["cap"], slopes=s["slopes"], positions=s["positions"])


def _run_own(s):
    from context_paged_attention_gb300 import binding as B

    c = s["case"]
    q, k = s["q"], s["k_new"]
    if c["op"] == "append" or c["append"]:
        B.cp_rope_kv_write(s["desc"], s["pool_k"], s["pool_v"], q, k, s["v_new"], s["positions"], s["qo"],
                           s["indptr"], s["indices"], s["cos_sin"], s["q_rot"], s["k_rot"],
                           rot_begin=c["rot_begin"], style=B.ROPE_PAIRS if c["style"] == "pairs" else B.ROPE_HALVES,
                           dev_status=s["status"])
        q, k = s["q_rot"], s["k_rot"]
    if c["op"] == "append":
        return _append_outputs(s, q, k)
    one = _decode(c) and not c["pad"]
    extra = {}
    if not _decode(c):
        B.own_token_attn(q, k, s["v_new"], s["qo"], c["rows"], s["max_new"], s["scale"], s["o_own"], s["lse_own"],
                         mod=s["mod"])
        extra = {"extra_o": s["o_own"], "extra_lse": s["lse_own"]}
    B.cp_paged_attn_fused(s["desc"], s["pool_k"], s["pool_v"], q, s["kv_len"], s["max_kv"], s["indptr"],
                          s["indices"], s["scale"], s["out"], s["ws"], lse_out=s["lse"],
                          qo_indptr=None if one else s["qo"], num_rows=c["rows"], row_order=s["order"],
                          dev_status=s["status"], mod=s["mod"], **extra)
    return {"out": s["out"], "lse": s["lse"]}


def _append_outputs(s, q, k):
    out = {"q": q, "k": k}
    for name in ("pool_k", "pool_v"):
        x = s[name]
        if x is not None:
            out[name] = x.view(torch.float8_e4m3fn) if s["case"]["pool"] == "e4m3" else x
    return out


# ---- the plain forms

def _rotate(s, x):
    """Rows x [t, h, d] rotated by their positions, in 32 bits (padding rows come out as anything)."""
    c = s["case"]
    r, b = c["rot"], c["rot_begin"]
    cs = s["cos_sin"][s["positions"].clamp(min=0).long()].unsqueeze(1)
    cos, sin = cs[..., : r // 2], cs[..., r // 2:]
    x = x.float()
    seg = x[..., b: b + r]
    u, v = (seg[..., : r // 2], seg[..., r // 2:]) if c["style"] == "halves" else (seg[..., 0::2], seg[..., 1::2])
    a, e = u * cos - v * sin, v * cos + u * sin
    turned = torch.cat([a, e], -1) if c["style"] == "halves" else torch.stack([a, e], -1).flatten(-2)
    return torch.cat([x[..., :b], turned, x[..., b + r:]], -1)


def _slot_rows(s, row, pos):
    """Pool row of head 0 .. hkv - 1 holding position pos of each row: [..., hkv]."""
    c = s["case"]
    psl = c["page"] // c["p"]
    last = s["indices"].numel() - 1
    page = s["indices"][(s["indptr"][row].long() + pos // c["page"]).clamp(max=last)].long()
    off = pos % c["page"]
    run = off // c["il"]
    slot = run // c["p"] * c["il"] + off % c["il"]
    heads = torch.arange(c["hkv"], device="cuda")
    return (((run % c["p"]) * s["n_pages"] + page)[..., None] * c["hkv"] + heads) * psl + slot[..., None]


def _append(s):
    c = s["case"]
    real = s["positions"] >= 0
    q, k = _rotate(s, s["q"]), _rotate(s, s["k_new"])
    s["q_rot"] = torch.where(real[:, None, None], q.to(s["q"].dtype), s["q_rot"])
    s["k_rot"] = torch.where(real[:, None, None], k.to(s["q"].dtype), s["k_rot"])
    used = s["k_new"].shape[0] - c["pad"]
    pos = s["positions"][:used].long()
    row = torch.searchsorted(s["qo"][1:].contiguous(), torch.arange(used, device="cuda", dtype=torch.int32),
                             right=True)
    at = _slot_rows(s, row, pos).flatten()
    _put(s, "pool_k", at, k[:used].flatten(0, 1), s["kd"])
    if s["pool_v"] is not None:
        _put(s, "pool_v", at, s["v_new"][:used].float().flatten(0, 1), s["vd"])


def _put(s, name, at, x, descale):
    c, pool, d = s["case"], s[name], x.shape[-1]
    if c["pool"] == "fp4":
        n = _pool_rows(c, s["n_pages"])
        codes, sf = _fp4_rows(x, descale)
        pool[: n * d // 2].view(n, d // 2)[at] = codes
        pool[n * d // 2:].view(n, d // 16)[at] = sf
    elif c["pool"] == "e4m3":
        pool.view(-1, d)[at] = _e4m3_bytes(x / descale)
    else:
        pool.view(-1, d)[at] = x.to(pool.dtype)


def _get(s, name, at, descale):
    """Values of pool rows `at`, in 32 bits."""
    c, pool, d = s["case"], s[name], s["case"]["d"]
    if c["pool"] == "fp4":
        n = _pool_rows(c, s["n_pages"])
        codes = pool[: n * d // 2].view(n, d // 2)[at]
        sf = pool[n * d // 2:].view(n, d // 16)[at].view(torch.float8_e4m3fn).float()
        v = torch.index_select(s["pairs"], 0, codes.flatten().int()).view(*codes.shape[:-1], -1, 16)
        return (v * (sf * descale).unsqueeze(-1)).flatten(-2)
    if c["pool"] == "e4m3":
        return pool.view(-1, d)[at].view(torch.float8_e4m3fn).float() * descale
    return pool.view(-1, d)[at].float()


def _attend(s, q, k_new):
    c = s["case"]
    b, h, g, d, m = c["rows"], c["hkv"], c["hq"] // c["hkv"], c["d"], s["max_new"]
    used = q.shape[0] - c["pad"]
    rows = torch.arange(b, device="cuda")
    span = s["qo"][1:] - s["qo"][:-1]
    i = torch.arange(m, device="cuda")
    mine = i < span[:, None]                                      # [b, m]: token i of row b is one
    tok = (s["qo"][:-1, None] + i).clamp(max=max(used - 1, 0)).long()
    # queries [b, h, m * g, d]; keys and values [b, h, keys, d]
    qs = q[tok].float().view(b, m, h, g, d).permute(0, 2, 1, 3, 4).reshape(b, h, m * g, d)
    pos = torch.arange(s["max_kv"], device="cuda").expand(b, -1)
    at = _slot_rows(s, rows[:, None], pos)
    k = _get(s, "pool_k", at, s["kd"]).transpose(1, 2)
    v = _get(s, "pool_v", at, s["vd"]).transpose(1, 2)
    seen = (pos < s["kv_len"][:, None])[:, None, :].expand(b, m, -1)
    qpos = s["positions"][tok]                                    # [b, m]
    kpos = pos
    if not _decode(c):  # the row's own new tokens, causally
        k = torch.cat([k, k_new[tok].float().transpose(1, 2)], 2)
        v = torch.cat([v, s["v_new"][tok].float().transpose(1, 2)], 2)
        seen = torch.cat([seen, (i[None, :] <= i[:, None]) & mine[:, None, :]], 2)
        kpos = torch.cat([kpos, qpos], 1)
    sc = torch.matmul(qs, k.transpose(2, 3)).view(b, h, m, g, -1) * s["scale"]
    if c["cap"]:
        sc = c["cap"] * torch.tanh(sc / c["cap"])
    if s["slopes"] is not None:
        away = (kpos[:, None, :] - qpos[:, :, None]).float()      # [b, m, keys]
        sc = sc + s["slopes"].view(h, 1, g, 1) * away[:, None, :, None, :]
    sc = sc.masked_fill(~(seen & mine[..., None])[:, None, :, None, :], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = torch.exp(sc - top)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(b, h, m * g, -1), v).view(b, h, m, g, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 2, 1, 3, 4).reshape(b, m, h * g, d)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(b, m, h * g)
    out = torch.zeros_like(q)
    out_lse = torch.full(q.shape[:2], -math.inf, device="cuda")
    out[tok[mine]] = o[mine].to(q.dtype)
    out_lse[tok[mine]] = lse[mine]
    return {"out": out, "lse": out_lse}


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    q, k = s["q"], s["k_new"]
    if c["op"] == "append" or c["append"]:
        _append(s)
        q, k = s["q_rot"], s["k_rot"]
    if c["op"] == "append":
        return _append_outputs(s, q, k)
    return _attend(s, q, k)


# ---- the definitions in 64 bits, row by row and partner by partner

def _exact_e4m3(x):
    """Nearest E4M3 value (ties to the even code), magnitudes past 448 at 448."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.copysign(torch.round(a / step) * step, x).clamp(-448.0, 448.0)


def _exact_fp4(x, descale):
    """Values that 4-bit rows x are stored as."""
    v = (x / descale).unflatten(-1, (-1, 16))
    s = _exact_e4m3(v.abs().amax(-1, keepdim=True) / 6.0)
    a = torch.where(s > 0, v.abs() / s, torch.zeros_like(v)).clamp(max=6.0)
    e = torch.floor(torch.log2(a.clamp(min=1.0)))
    step = torch.exp2(e - 1)
    return (torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v) * s * descale).flatten(-2)


def _exact_stored(c, x, descale):
    if c["pool"] == "fp4":
        return _exact_fp4(x, descale)
    if c["pool"] == "e4m3":
        return _exact_e4m3(x / descale) * descale
    return x.to(torch.float32 if c["pool"] == "fp32" else torch.bfloat16).double()


def _exact_turn(s, x):
    """Rotation as a product of complex numbers; positions from the cos / sin table given."""
    c = s["case"]
    r, b = c["rot"], c["rot_begin"]
    cs = s["cos_sin"].double()[s["positions"].clamp(min=0).long()]
    z = torch.complex(cs[:, : r // 2], cs[:, r // 2:])[:, None, :]
    y = x.double().clone()
    seg = y[..., b: b + r]
    if c["style"] == "pairs":
        w = torch.complex(seg[..., 0::2].contiguous(), seg[..., 1::2].contiguous()) * z
        seg[..., 0::2], seg[..., 1::2] = w.real, w.imag
    else:
        w = torch.complex(seg[..., : r // 2].contiguous(), seg[..., r // 2:].contiguous()) * z
        seg[..., : r // 2], seg[..., r // 2:] = w.real.clone(), w.imag.clone()
    return y


def _partner_offsets(c, p):
    return [o for o in range(c["page"]) if o // c["il"] % c["p"] == p]


def _exact_values(s, name):
    """Every pool row's value in 64 bits, as [p, pages, hkv, page / p, d]."""
    c, d = s["case"], s["case"]["d"]
    pool, descale = s[name], s["kd"] if name == "pool_k" else s["vd"]
    shape = (c["p"], s["n_pages"], c["hkv"], c["page"] // c["p"], d)
    if c["pool"] == "fp4":
        n = _pool_rows(c, s["n_pages"])
        b = pool[: n * d // 2].view(n, d // 2).to(torch.int16)
        nib = torch.stack([b & 15, b >> 4], -1).flatten(1)
        mant, ex = (nib & 1).float(), (nib >> 1) & 3
        mag = torch.where(ex == 0, 0.5 * mant, (1 + 0.5 * mant) * torch.exp2(ex.float() - 1))
        mag = torch.where(nib > 7, -mag, mag)
        sf = pool[n * d // 2:].view(n, d // 16).view(torch.float8_e4m3fn).float()
        # exact in 32 bits: at most six significant bits
        return (mag.unflatten(-1, (-1, 16)) * sf[..., None]).flatten(-2).view(shape), descale
    if c["pool"] == "e4m3":
        return pool.view(torch.float8_e4m3fn).float().view(shape), descale
    return pool.view(shape), 1.0


def _exact_context(s, vals, b, n):
    """First n positions of row b in order, [n, hkv, d] in 64 bits."""
    c = s["case"]
    v, descale = vals
    pages = s["indices"][int(s["indptr"][b]): int(s["indptr"][b + 1])].long()[: -(-n // c["page"])]
    out = torch.empty(len(pages), c["page"], c["hkv"], c["d"], dtype=torch.float64, device="cuda")
    for p in range(c["p"]):
        out[:, _partner_offsets(c, p)] = v[p][pages].transpose(1, 2).double()
    return out.flatten(0, 1)[:n] * descale


def exact(c, seed):
    if c["op"] == "attend" and c["rows"] * c["ctx_hi"] * c["hkv"] * c["d"] > 4e9:
        return None
    s = prepare(c, seed)
    layer = s["q"].dtype
    new, _ = _lengths(c)
    used = sum(new)
    q, k = s["q"].double(), s["k_new"].double()
    qo = s["qo"].tolist()
    if c["op"] == "append" or c["append"]:
        q, k = _exact_turn(s, s["q"]), _exact_turn(s, s["k_new"])
        stored = _exact_stored(c, k, s["kd"])
        stored_v = None if s["v_new"] is None else _exact_stored(c, s["v_new"].double(), s["vd"])
    if c["op"] == "append":
        q[used:], k[used:] = 0, 0
        out = {"q": q, "k": k}
        for name, rows in (("pool_k", stored if c["pool"] == "e4m3" else k), ("pool_v", stored_v)):
            if s[name] is None:
                continue
            kd = s["kd"] if name == "pool_k" else s["vd"]
            pool = s[name].view(torch.float8_e4m3fn).float().double() if c["pool"] == "e4m3" else s[name].double()
            place = {o: (p, i) for p in range(c["p"]) for i, o in enumerate(_partner_offsets(c, p))}
            positions, first, pages = s["positions"].tolist(), s["indptr"].tolist(), s["indices"].tolist()
            for b in range(c["rows"]):
                for t in range(qo[b], qo[b + 1]):
                    p, slot = place[positions[t] % c["page"]]
                    page = pages[first[b] + positions[t] // c["page"]]
                    pool[p, page, :, slot] = rows[t] / (kd if c["pool"] == "e4m3" else 1.0)
            out[name] = pool
        return out
    if c["append"]:
        q, k = q.to(layer).double(), k.to(layer).double()
    vals_k, vals_v = _exact_values(s, "pool_k"), _exact_values(s, "pool_v")
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    g = c["hq"] // c["hkv"]
    kv_len = s["kv_len"].tolist()
    for b in range(c["rows"]):
        lo, hi, n = qo[b], qo[b + 1], kv_len[b]
        ks, vs = _exact_context(s, vals_k, b, n), _exact_context(s, vals_v, b, n)
        if _decode(c):
            if c["append"]:
                ks[-1], vs[-1] = stored[lo], stored_v[lo]
        else:
            ks, vs = torch.cat([ks, k[lo:hi]]), torch.cat([vs, s["v_new"][lo:hi].double()])
        qpos = s["positions"][lo:hi].double()
        kpos = torch.arange(ks.shape[0], device="cuda", dtype=torch.float64)
        for h in range(c["hkv"]):
            sc = torch.einsum("mgd,ld->mgl", q[lo:hi, h * g: (h + 1) * g], ks[:, h]) * s["scale"]
            if c["cap"]:
                sc = c["cap"] * torch.tanh(sc / c["cap"])
            if s["slopes"] is not None:
                sc = sc + s["slopes"][h * g: (h + 1) * g].double()[None, :, None] * (
                    kpos[None, None, :] - qpos[:, None, None])
            sc = sc.masked_fill((kpos[None, :] > qpos[:, None])[:, None, :], -math.inf)
            lse[lo:hi, h * g: (h + 1) * g] = torch.logsumexp(sc, -1)
            out[lo:hi, h * g: (h + 1) * g] = torch.softmax(sc, -1) @ vs[:, h]
    return {"out": out, "lse": lse}
