"""Rotated appends, 4-bit pools and modified scores on the GPU against the
float64 oracle.

Attention is checked against the pool's own bytes (decoded by the oracle) and
the queries the calls took; what the bytes should be is checked apart.  Bars:
  * P V with probabilities in float16 (one-token rows over 4-bit pools, and over
    E4M3 pools with modified scores: the kernel over pools of codes): p~_k = p_k
    (1 + d_k) + a_k with |d_k| <= 2^-11 and, below 2^-14, |a_k| <= 2^-25 instead;
    the sum Z of the p_k is float32, so O~ - O = sum (p_k d_k + a_k) v_k / Z and
    |O~ - O| <= 2^-11 A + 2^-25 sum |v_k| / Z with A the weights applied to |V|.
    The running max is one of the scores or below the largest, so Z >= sum
    exp(s - max s) and the second term is at most 2^-25 B, B = sum |V| / sum
    exp(s - max s);
  * in bf16 (multi-token rows): 2^-8 relatively, normalised by the rounded sum:
    2 * 2^-8 A;
  * in float32 or as a 16-bit pair (the rest): 0;
  each plus 1e-4 A + 2e-5 for the float32 scores (a score is off by some 2^-20
  of its size, 2^-20 of the cap where capped, and a weight relatively by that
  much absolutely), and 2^-8 |O| for a bf16 output.
LSE: 1e-4 + 2^-20 |LSE|.  fp32 layers: 2e-6 A + 1e-5.
"""

import dataclasses

import numpy as np
import pytest
import torch

import oracle
from context_paged_attention_gb300 import workloads as W
from helpers import assert_close_lse, assert_within_bound, f64, raw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _att(w, **kw):
    from context_paged_attention_gb300.step import StripedAttention

    return StripedAttention(w, device="cuda", **kw)


def pool_values(att, value=False):
    """Pool contents as float64 [P, pages, H, slots, D], decoded by the oracle."""
    w, pool = att.w, att.pool_v if value else att.pool_k
    ds = w.v_descale if value else w.k_descale
    if w.kv_dtype == "fp4":
        codes, scales = (raw(x) for x in att.desc.fp4_views(pool, value))
        un = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
        return oracle.fp4_dequantize(un, scales, ds)
    if w.kv_dtype == "fp8":
        return oracle.e4m3_dequantize(raw(pool), float(np.float32(ds)))
    return f64(pool)


def row_values(w, pool, b, n):
    """First n positions of row b out of pool values: [n, H, D]."""
    pages = w.kv_page_indices[w.kv_page_indptr[b]: w.kv_page_indptr[b + 1]]
    out = np.empty((n, pool.shape[2], pool.shape[4]))
    for j in range(n):
        p, page, slot = oracle.placement(pages, j, w.page_size, w.P, w.interleave)
        out[j] = pool[p, page, :, slot]
    return out


def p_float16(w):
    """Whether one-token rows take the kernel over pools of codes, which rounds P to float16."""
    return w.kv_dtype == "fp4" or (w.kv_dtype == "fp8" and (w.softcap > 0 or w.slopes is not None))


def check_step(w, att, out, lse, heads=None, rows=None):
    """A step's merged output and LSE against the oracle over what the pool holds."""
    K, V = pool_values(att), pool_values(att, True)
    q, kn = f64(att.query), f64(att.k_rot if w.rot_dim else att.k_new)
    got_o, got_l = f64(out), lse.cpu().numpy().astype(np.float64)
    vn = f64(att.v_new)
    for b in range(w.num_real_rows) if rows is None else rows:
        n, c, t0 = int(w.kv_len[b]), int(w.ctx_len[b]), int(w.qo_indptr[b])
        ks, vs = row_values(w, K, b, n), row_values(w, V, b, n)
        for i in range(int(w.new_len[b])):
            t = t0 + i
            kk, vv = ks, vs
            if not w.decode:
                kk, vv = np.concatenate([ks, kn[t0: t + 1]]), np.concatenate([vs, vn[t0: t + 1]])
            O, L, A, Bd = oracle.modified_attention(q[t], kk, vv, w.scale, c + i, np.arange(len(kk)), w.softcap,
                                                    w.slopes)
            if w.dtype == "fp32":
                bound = 2e-6 * A + 1e-5
            else:
                pv = 2.0 ** -11 * A + 2.0 ** -25 * Bd if w.decode and p_float16(w) else 0.0
                if not w.decode:
                    pv = 2.0 ** -7 * A
                bound = pv + 1e-4 * A + 2e-5 + 2.0 ** -8 * np.abs(O)
            assert_within_bound(got_o[t], O, bound, f"O row {b} token {i}")
            assert_close_lse(got_l[t], L, 1e-4 + 2.0 ** -20 * np.abs(L[np.isfinite(L)]).max(initial=0.0),
                             f"LSE row {b} token {i}")
    t_end = int(w.qo_indptr[w.num_real_rows])
    assert np.all(got_o[t_end:] == 0) and np.all(got_l[t_end:] == -np.inf)


def bits(x):
    return x.view(np.uint32) if x.dtype == np.float32 else x


# ---------------------------------------------------------------- appends

def turned32(w, x, positions, tab):
    """Rows turned in float32, each product and sum rounded (the call's arithmetic)."""
    x = np.array(oracle.raw_to_f64(x).astype(np.float32), copy=True)
    r, h = tab.shape[1], tab.shape[1] // 2
    i = np.arange(h)
    a = w.rot_begin + (2 * i if w.rope_pairs else i)
    b = a + 1 if w.rope_pairs else a + h
    real = positions >= 0
    c, s = tab[positions[real], :h][:, None], tab[positions[real], h:][:, None]
    u, v = x[real][..., a], x[real][..., b]
    y = x[real]
    with np.errstate(all="ignore"):
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    x[real] = y
    return x


def layer_bits(w, x):
    return x if w.dtype == "fp32" else W.f32_to_bf16_bits(x)


def stored(w, x, descale):
    """What a pool of w holds for float32 rows x: (rows,) or (code bytes, scales)."""
    if w.kv_dtype == "fp4":
        codes, scales = oracle.fp4_quantize(x, descale)
        return oracle.fp4_pack(codes), scales
    if w.kv_dtype == "fp8":
        return (oracle.e4m3_quantize(x, descale),)
    return (layer_bits(w, x),)


def check_pool(w, att, value, rows, positions, qo, before):
    """Pool bytes: what `before` held, and `rows` (float32) of the tokens at their places."""
    pool = att.pool_v if value else att.pool_k
    now = att.desc.fp4_views(pool, value) if w.kv_dtype == "fp4" else (pool,)
    parts = stored(w, rows, w.v_descale if value else w.k_descale)
    for got, old, new in zip(now, before, parts):
        want = raw(old).copy()
        for b in range(len(qo) - 1):
            pages = w.kv_page_indices[w.kv_page_indptr[b]: w.kv_page_indptr[b + 1]]
            for t in range(qo[b], qo[b + 1]):
                if positions[t] >= 0:
                    p, page, slot = oracle.placement(pages, int(positions[t]), w.page_size, w.P, w.interleave)
                    want[p, page, :, slot] = new[t]
        assert np.array_equal(bits(raw(got)), bits(want)), "values" if value else "keys"


def _mixed(seed, hq, hkv, d, P, page, I=1, dtype="bf16", new=(1, 3, 17, 2), ctx=(5, 0, 40, 130), pad=(0, 2), T=None):
    w = W.build_workload("m", dtype=dtype, P=P, page_size=page, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                         decode=False, ctx_len=ctx, new_len=new, padding_spans=list(pad),
                         num_tokens=T if T is not None else sum(new) + sum(pad) + 3, seed=seed)
    return W.interleaved(w, I)


def _latent(seed):
    return W.build_workload("l", dtype="bf16", P=4, page_size=64, num_q_heads=16, num_kv_heads=1, head_dim=576,
                            head_dim_v=512, mla=True, decode=False, scale=0.07, ctx_len=[3, 0, 100],
                            new_len=[1, 20, 5], padding_spans=[2], num_tokens=32, seed=seed)


APPENDS = {
    "halves_bf16": lambda: W.rotated(_mixed(1, 32, 8, 128, 4, 16), 128),
    "pairs_bf16_part": lambda: W.rotated(_mixed(2, 8, 8, 128, 4, 16, I=4), 64, 64, pairs=True),
    "halves_d64_front": lambda: W.rotated(_mixed(3, 4, 1, 64, 2, 16, I=4), 32),
    "odd_width": lambda: W.rotated(_mixed(4, 4, 2, 128, 1, 8), 106, 22, pairs=True),
    "odd_start_halves": lambda: W.rotated(_mixed(5, 4, 2, 64, 8, 8), 10, 3),
    "odd_start_pairs": lambda: W.rotated(_mixed(6, 4, 2, 64, 8, 8), 50, 13, pairs=True),
    "two_values": lambda: W.rotated(_mixed(7, 1, 1, 64, 1, 1), 2, 62),
    "fp32": lambda: W.rotated(_mixed(8, 4, 1, 64, 2, 16, dtype="fp32"), 64),
    "fp32_odd": lambda: W.rotated(_mixed(9, 2, 2, 20, 2, 4, dtype="fp32"), 14, 5),
    "e4m3": lambda: W.fp8_pool(W.rotated(_mixed(10, 16, 8, 128, 8, 64), 128, pairs=True), 0.0123, 0.0137),
    "e4m3_odd": lambda: W.fp8_pool(W.rotated(_mixed(11, 2, 1, 64, 2, 4), 30, 9), 0.0123, 0.0137),
    "fp4": lambda: W.fp4_pool(W.rotated(_mixed(12, 32, 8, 128, 4, 16), 128), 0.0021, 0.0023),
    "fp4_pairs": lambda: W.fp4_pool(W.rotated(_mixed(13, 8, 2, 64, 4, 16, I=2), 32, 32, pairs=True), 0.0021, 0.0023),
    "fp4_odd": lambda: W.fp4_pool(W.rotated(_mixed(14, 8, 2, 64, 1, 2), 34, 7), 0.0021, 0.0023),
    "fp4_half_block": lambda: W.fp4_pool(W.rotated(_mixed(18, 8, 2, 128, 2, 8), 48, 8), 0.0021, 0.0023),
    "latent": lambda: W.rotated(_latent(15), 64, 512, pairs=True),
    "latent_halves": lambda: W.rotated(_latent(16), 64, 512),
    "wide_head": lambda: W.rotated(_mixed(17, 2, 1, 96, 2, 4), 96),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", sorted(APPENDS))
def test_rope_write(name, in_place):
    from context_paged_attention_gb300 import binding as B
    from context_paged_attention_gb300.step import rope_table

    w = APPENDS[name]()
    att = _att(w)
    pools = [(False, att.pool_k)] + ([] if w.mla else [(True, att.pool_v)])
    before = {v: tuple(x.clone() for x in (att.desc.fp4_views(p, v) if w.kv_dtype == "fp4" else (p,)))
              for v, p in pools}
    # the history went in through the same call, keys only; the tables hold its rows
    tab = rope_table(att.cos_sin.shape[0], w.rot_dim, w.rope_base)
    q, k = att.q.clone(), att.k_new.clone()
    mark = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    q_out, k_out = (q, k) if in_place else mark
    B.cp_rope_kv_write(att.desc, att.pool_k, att.pool_v, q, k, att.v_new, att.positions, att.qo_indptr,
                       att.page_indptr, att.page_indices, att.cos_sin, q_out, k_out, rot_begin=w.rot_begin,
                       style=att.rope_style, dev_status=att.dev_status)
    torch.cuda.synchronize()
    assert att.status() == 0
    real = w.positions >= 0
    for x, got, old in ((w.q, q_out, w.q), (w.k_new, k_out, w.k_new)):
        y = turned32(w, x, w.positions, tab)
        assert np.array_equal(bits(raw(got))[real], bits(layer_bits(w, y))[real])
        rest = raw(got)[~real]  # padding rows as they were
        assert np.array_equal(bits(rest), bits(old[~real])) if in_place else np.all(oracle.raw_to_f64(rest) == 7.0)
        # and against the definition: three float32 roundings of the terms, one to the output
        x64 = oracle.raw_to_f64(x)[real]
        want = oracle.rotate(x64, w.positions[real], tab, w.rot_begin, att.rope_style)
        u = 0.0 if w.dtype == "fp32" else 2.0 ** -8
        size = np.abs(x64).max(axis=-1, keepdims=True)
        assert_within_bound(oracle.raw_to_f64(raw(got))[real], want, u * np.abs(want) + 1.01 * 6 * 2.0 ** -24 * size + 1e-30)
    qo = w.qo_indptr[: w.num_real_rows + 1]
    check_pool(w, att, False, turned32(w, w.k_new, w.positions, tab), w.positions, qo, before[False])
    if not w.mla:
        check_pool(w, att, True, oracle.raw_to_f64(w.v_new).astype(np.float32), w.positions, qo, before[True])


@pytest.mark.parametrize("kv", ["same", "fp8", "fp4"])
def test_rope_write_is_rotation_then_kv_write(kv):
    """Position 0 rotates by nothing: the call then writes what cp_kv_write writes, bit for bit."""
    w = _mixed(20, 8, 2, 64, 2, 8, new=(1, 1, 1), ctx=(0, 0, 0))
    w = {"same": lambda x: x, "fp8": lambda x: W.fp8_pool(x, 0.0123, 0.0137),
         "fp4": lambda x: W.fp4_pool(x, 0.0021, 0.0023)}[kv](w)
    plain, turned = _att(w), _att(W.rotated(w, 64))
    plain.write_new()
    turned.write_new()
    torch.cuda.synchronize()
    assert torch.equal(plain.pool_k.view(torch.uint8), turned.pool_k.view(torch.uint8))
    assert torch.equal(plain.pool_v.view(torch.uint8), turned.pool_v.view(torch.uint8))
    n = int(w.qo_indptr[w.num_real_rows])
    assert torch.equal(turned.k_rot[:n], turned.k_new[:n])


def test_rope_write_bad_places_are_reported():
    """A position past the rotation table skips its token whole; a rejected page only its pool rows."""
    w = W.rotated(_mixed(21, 4, 2, 64, 2, 8, new=(2, 2, 2), ctx=(3, 9, 20)), 64)
    att = _att(w)
    pos = att.positions.clone()
    pos[3] = att.cos_sin.shape[0]  # row 1's second token
    pool = att.pool_k.clone(), att.pool_v.clone()
    att.positions = pos
    att.q_rot.fill_(7.0)
    att.k_rot.fill_(7.0)
    att.write_new()
    torch.cuda.synchronize()
    assert att.status() == 5  # CPATTN_DEV_POS_PAST_ROPE
    assert torch.all(att.q_rot[3] == 7) and torch.all(att.k_rot[3] == 7) and not torch.any(att.q_rot[2] == 7)
    ref = _att(w)
    ref.write_new()
    torch.cuda.synchronize()
    p, page, slot = oracle.placement(w.kv_page_indices[w.kv_page_indptr[1]:], 10, 8, 2)
    for got, old, full in ((att.pool_k, pool[0], ref.pool_k), (att.pool_v, pool[1], ref.pool_v)):
        want = full.clone()
        want[p, page, :, slot] = old[p, page, :, slot]
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    # a page outside the pool: reported, the rotated rows are there all the same
    att = _att(w)
    idx = att.page_indices.clone()
    idx[int(w.kv_page_indptr[2]) + 20 // 8] = w.num_pages + 5
    att.page_indices = idx
    att.write_new()
    torch.cuda.synchronize()
    assert att.status() == 1
    assert torch.equal(att.q_rot[:6], ref.q_rot[:6]) and torch.equal(att.k_rot[:6], ref.k_rot[:6])


def test_fp4_write_special_values():
    """Zeros (both signs), NaN, infinities, values below the smallest scale and past the largest."""
    from context_paged_attention_gb300 import binding as B

    w = W.fp4_pool(_mixed(22, 2, 1, 64, 1, 4, new=(8,), ctx=(0,), pad=(), T=8), 0.25, 4.0)
    att = _att(w)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((8, 1, 64)).astype(np.float32)
    x[1, 0, :16] = 0.0
    x[1, 0, 16:32] = -0.0
    x[2, 0, 5] = np.nan
    x[3, 0, 7] = np.inf
    x[3, 0, 40] = -np.inf
    x[4] *= 1e-4
    x[5] *= 1e6
    x[6, 0, ::16] *= 1e3
    x[7] = np.tile(np.array([6, 5, -5, 3.5, 2.5, 1.75, 1.25, .75, .25, -.25, -.75, 0, 1, 2, 4, -3.5], np.float32), 4)
    b = W.f32_to_bf16_bits(np.where(np.isnan(x), 0, x))
    b[np.isnan(x)] = 0x7FC0
    t = torch.from_numpy(b.view(np.int16)).view(torch.bfloat16).cuda()
    B.cp_kv_write(att.desc, att.pool_k, att.pool_v, t, t, att.positions, att.qo_indptr, att.page_indptr,
                  att.page_indices, dev_status=att.dev_status)
    torch.cuda.synchronize()
    for value, ds in ((False, 0.25), (True, 4.0)):
        pool = att.pool_v if value else att.pool_k
        codes, scales = (raw(v) for v in att.desc.fp4_views(pool, value))
        want_c, want_s = oracle.fp4_quantize(oracle.raw_to_f64(b).astype(np.float32), ds)
        want_c = oracle.fp4_pack(want_c)
        for j in range(8):
            p, page, slot = oracle.placement(w.kv_page_indices, j, w.page_size, w.P)
            assert np.array_equal(scales[p, page, :, slot], want_s[j]), j
            assert np.array_equal(codes[p, page, :, slot], want_c[j]), j


# ---------------------------------------------------------------- attention

SLOPES = lambda h: (2.0 ** (-8.0 * (np.arange(h) + 1) / h)).astype(np.float32)  # noqa: E731


def _decode(seed, hq, hkv, d, P, page, ctx, I=1, pad=None, dtype="bf16", qs=1.0):
    w = W.build_workload("d", dtype=dtype, P=P, page_size=page, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                         ctx_len=ctx, new_len=[1] * len(ctx), padding_spans=pad, seed=seed)
    return W.interleaved(_spread(w, qs), I)


def _spread(w, qs):
    """Queries spread by qs (exact powers of two)."""
    if qs == 1.0:
        return w
    q = oracle.raw_to_f64(w.q) * qs
    return dataclasses.replace(w, q=q.astype(np.float32) if w.dtype == "fp32" else W.f32_to_bf16_bits(
        np.nan_to_num(q, nan=0.0).astype(np.float32)))


F4 = lambda w: W.fp4_pool(w, 0.0021, 0.0023)  # noqa: E731
F8 = lambda w: W.fp8_pool(w, 0.0123, 0.0137)  # noqa: E731
STEPS = {
    # 4-bit pools, one token a row: groups 1 .. 16, both widths, page runs of 1 to 64 rows, empty stripes
    "fp4_g4": lambda: F4(_decode(30, 32, 8, 128, 4, 16, [700, 0, 1, 31, 32, 33, 2500])),
    "fp4_g1_d64": lambda: F4(_decode(31, 4, 4, 64, 2, 8, [3, 400, 1])),
    "fp4_g2_d64": lambda: F4(_decode(32, 4, 2, 64, 8, 64, [3, 400, 130], I=4)),
    "fp4_g8": lambda: F4(_decode(33, 16, 2, 128, 8, 64, [5, 900, 129])),
    "fp4_g16": lambda: F4(_decode(34, 16, 1, 128, 1, 16, [5, 900, 127], I=2)),
    "fp4_g16_d64": lambda: F4(_decode(35, 32, 2, 64, 2, 2, [5, 300, 64])),
    "fp4_one_slot_pages": lambda: F4(_decode(36, 8, 2, 128, 4, 4, [5, 300, 64])),
    "fp4_odd_page": lambda: F4(_decode(37, 8, 2, 128, 2, 6, [5, 301, 64], I=3)),
    "fp4_split": lambda: F4(_decode(38, 4, 1, 128, 1, 64, [5000, 20, 2047, 2048, 4096])),
    "fp4_padded": lambda: F4(_decode(39, 8, 2, 128, 4, 16, [40, 300], pad=[1, 0, 2])),
    "fp4_spread": lambda: F4(_decode(40, 8, 2, 128, 2, 16, [40, 900], qs=8.0)),
    # 4-bit pools, several tokens a row
    "fp4_mixed": lambda: F4(_mixed(41, 8, 2, 128, 4, 16, new=(1, 40, 2, 9), ctx=(300, 0, 700, 33))),
    "fp4_mixed_d64_g16": lambda: F4(_mixed(42, 16, 1, 64, 2, 8, I=2, new=(3, 1, 17, 20), ctx=(0, 5, 40, 300))),
    "fp4_mixed_g1_split": lambda: F4(_mixed(43, 2, 2, 128, 1, 16, new=(5, 1), ctx=(2500, 2100))),
    # modified scores: every kernel that forms scores
    "cap_bf16": lambda: W.scored(_decode(50, 8, 2, 128, 4, 16, [700, 0, 33], qs=8.0), 20.0),
    "slopes_bf16": lambda: W.scored(_decode(51, 8, 2, 64, 4, 16, [700, 1, 33], I=2), 0.0, SLOPES(8)),
    "both_e4m3": lambda: W.scored(F8(_decode(52, 16, 2, 128, 8, 64, [700, 2, 33], qs=4.0)), 30.0, SLOPES(16)),
    "both_g16": lambda: W.scored(_decode(53, 16, 1, 128, 2, 16, [700, 0, 33], I=4, qs=4.0), 15.0, SLOPES(16)),
    "both_g16_e4m3": lambda: W.scored(F8(_decode(54, 16, 1, 64, 2, 16, [700, 0, 33], qs=4.0)), 15.0, SLOPES(16)),
    "both_fp4": lambda: W.scored(F4(_decode(55, 8, 2, 128, 4, 16, [700, 0, 2500], I=2, qs=4.0)), 15.0, SLOPES(8)),
    "both_fp4_g16": lambda: W.scored(F4(_decode(56, 16, 1, 64, 2, 16, [700, 0, 33], qs=4.0)), 15.0, SLOPES(16)),
    "both_fp32": lambda: W.scored(_decode(57, 4, 1, 64, 2, 16, [36, 99, 600], dtype="fp32", qs=4.0), 20.0, SLOPES(4)),
    "slopes_fp32_I": lambda: W.scored(_decode(58, 8, 1, 128, 2, 16, [36, 99], I=4, dtype="fp32"), 0.0, SLOPES(8)),
    "padded": lambda: W.scored(_decode(59, 8, 2, 128, 4, 16, [40, 300], pad=[1, 0, 2]), 10.0, SLOPES(8)),
    "split": lambda: W.scored(_decode(60, 4, 1, 128, 1, 64, [5000, 2047]), 0.0, SLOPES(4)),
    "steep": lambda: W.scored(_decode(61, 4, 1, 128, 1, 64, [3000, 20]), 5.0, np.array([3, 0.5, -0.001, 0], np.float32)),
    "mixed": lambda: W.scored(_spread(_mixed(62, 8, 2, 128, 4, 16, new=(1, 40, 2, 9), ctx=(300, 0, 700, 33)), 4.0),
                              20.0, SLOPES(8)),
    "mixed_e4m3": lambda: W.scored(F8(_mixed(63, 4, 2, 64, 2, 8, I=2, new=(1, 40), ctx=(300, 150))), 2.0, SLOPES(4)),
    "mixed_fp4": lambda: W.scored(F4(_mixed(64, 16, 1, 128, 2, 8, new=(5, 1, 20), ctx=(300, 20, 0))), 2.0, SLOPES(16)),
    "mixed_fp32": lambda: W.scored(_mixed(65, 4, 2, 64, 2, 8, dtype="fp32", new=(1, 9), ctx=(300, 15)), 2.0, SLOPES(4)),
    "mixed_split": lambda: W.scored(_mixed(66, 4, 1, 128, 1, 16, new=(5, 1), ctx=(2500, 2100)), 0.0, SLOPES(4)),
    # more blocks of tokens than SMs: pieces in equal parts, several items a CTA, cut and whole ones
    "mixed_many": lambda: W.scored(_spread(_mixed(67, 32, 2, 64, 4, 16, new=(1, 300, 2, 17, 1, 250, 16, 33),
                                                  ctx=(900, 2500, 2500, 0, 3, 1100, 40, 700)), 4.0), 20.0, SLOPES(32)),
    "mixed_many_e4m3": lambda: W.scored(F8(_mixed(68, 32, 4, 128, 2, 32, I=2, new=(290, 1, 2, 33, 250, 64),
                                                  ctx=(2100, 700, 2049, 5, 1, 333))), 0.0, SLOPES(32)),
    # as a layer runs them: rotation on the way in, 4-bit pool, modified scores
    "layer_decode": lambda: W.scored(F4(W.rotated(_decode(70, 8, 2, 128, 4, 16, [700, 0, 33]), 128)), 30.0, SLOPES(8)),
    "layer_mixed": lambda: W.scored(F4(W.rotated(_mixed(71, 8, 2, 128, 4, 16), 64, 64, pairs=True)), 30.0, SLOPES(8)),
    "layer_plain": lambda: W.rotated(_decode(72, 8, 2, 64, 4, 16, [70, 0, 33], pad=[1]), 64),
    "layer_fp32": lambda: W.rotated(_mixed(73, 4, 1, 64, 2, 16, dtype="fp32"), 64),
}


@pytest.fixture(scope="module", params=sorted(STEPS))
def step(request):
    w = STEPS[request.param]()
    att = _att(w)
    att.run_step()
    torch.cuda.synchronize()
    assert att.status() == 0
    return w, att


def test_step(step):
    w, att = step
    check_step(w, att, att.out, att.lse)


def test_fused_step(step):
    w, att = step
    out, lse = torch.full_like(att.out, 7.0), torch.full_like(att.lse, 7.0)
    att.run_step_fused(out=out, lse=lse)
    torch.cuda.synchronize()
    assert att.status() == 0
    check_step(w, att, out, lse)


def test_partials(step):
    """One-token rows over 4-bit pools and modified scores: every partner's own partial."""
    w, att = step
    if not w.decode:
        pytest.skip("merged outputs cover multi-token rows")
    att.run_step()
    torch.cuda.synchronize()
    K, V = pool_values(att), pool_values(att, True)
    q = f64(att.query)
    for b in range(w.num_real_rows):
        n, t = int(w.kv_len[b]), int(w.qo_indptr[b])
        ks, vs = row_values(w, K, b, n), row_values(w, V, b, n)
        for p in range(w.P):
            idx = oracle.stripe_positions(n, w.P, p, w.interleave)
            O, L, A, Bd = oracle.modified_attention(q[t], ks[idx], vs[idx], w.scale, n - 1, idx, w.softcap, w.slopes)
            pv = 2.0 ** -11 * A + 2.0 ** -25 * Bd if p_float16(w) else 0.0
            bound = 2e-6 * A + 1e-5 if w.dtype == "fp32" else pv + 1e-4 * A + 2e-5
            assert_within_bound(att.o_parts[p, t].cpu().numpy(), O, bound, f"O row {b} partner {p}")
            assert_close_lse(att.lse_parts[p, t].cpu().numpy(), L,
                             1e-4 + 2.0 ** -20 * np.abs(L[np.isfinite(L)]).max(initial=0.0), f"LSE row {b} partner {p}")


def test_tp_and_graph(step):
    """The tensor-parallel head layout, and the step captured and replayed."""
    w, att = step
    out, lse = torch.empty_like(att.out), torch.empty_like(att.lse)
    if w.num_q_heads % w.P == 0:
        att.run_step_tp(out=out, lse=lse)
        torch.cuda.synchronize()
        check_step(w, att, out, lse)
    att.capture(fused=True)
    o1, l1 = (x.clone() for x in att.run_step_fused())
    att.out.fill_(7.0)
    o, l_ = att.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o1) and torch.equal(l_, l1)


def test_positions_default_matches_given():
    """Distances from kv_len (no positions passed) equal those from the step's positions."""
    from context_paged_attention_gb300 import binding as B

    for w in (STEPS["slopes_bf16"](), W.scored(_mixed(80, 8, 2, 128, 4, 16), 0.0, SLOPES(8)), STEPS["slopes_fp32_I"]()):
        att = _att(w)
        a = [x.clone() for x in att.run_step()]
        att.mod = B.score_mod(w.softcap, att.mod.tensors[0])
        b = att.run_step()
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_nothing_to_modify_is_the_plain_call():
    from context_paged_attention_gb300 import binding as B

    w = _decode(81, 8, 2, 128, 4, 16, [700, 3])
    att = _att(w)
    a = [x.clone() for x in att.run_step()]
    att.mod = B.score_mod(0.0)
    b = att.run_step()
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rejected_pages_leave_their_keys_out():
    """A page outside the pool is reported and its keys are left out -- at the start, middle and end of a row."""
    for kind in ("fp4_g4", "both_fp4", "both_g16", "both_e4m3", "mixed_fp4"):
        w = STEPS[kind]()
        b = int(np.argmax(w.kv_len))
        npg = int(w.kv_page_indptr[b + 1] - w.kv_page_indptr[b])
        for hit in (0, npg // 2):
            att = _att(w)
            att.write_new()
            idx = att.page_indices.clone()
            idx[int(w.kv_page_indptr[b]) + hit] = w.num_pages + 9
            att.page_indices = idx
            att.partial()
            torch.cuda.synchronize()
            assert att.status() == 1
            K, V = pool_values(att), pool_values(att, True)
            n, t = int(w.kv_len[b]), int(w.qo_indptr[b])
            ks, vs = row_values(w, K, b, n), row_values(w, V, b, n)
            for p in range(w.P):
                pos = oracle.stripe_positions(n, w.P, p, w.interleave)
                pos = pos[pos // w.page_size != hit]
                qpos = int(w.positions[t])
                O, L, A, Bd = oracle.modified_attention(f64(att.query)[t], ks[pos], vs[pos], w.scale, qpos, pos,
                                                        w.softcap, w.slopes)
                assert_within_bound(att.o_parts[p, t].cpu().numpy(), O,
                                    2.0 ** -7 * A + 2.0 ** -25 * Bd + 1e-4 * A + 2e-5, kind)
                assert_close_lse(att.lse_parts[p, t].cpu().numpy(), L, 2e-4, kind)


SHORT_TABLES = {
    "fp4": lambda: F4(_decode(90, 8, 2, 128, 4, 16, [63, 700, 31])),
    "e4m3_scored": lambda: W.scored(F8(_decode(91, 8, 2, 128, 4, 16, [63, 700, 31])), 20.0, SLOPES(8)),
    "fp4_mixed": lambda: F4(_mixed(92, 8, 2, 128, 4, 16, new=(4, 40), ctx=(60, 300))),
    "mixed_scored": lambda: W.scored(_mixed(93, 8, 2, 128, 4, 16, new=(4, 40), ctx=(60, 300)), 20.0, SLOPES(8)),
    "mixed_many": lambda: W.scored(_mixed(94, 32, 2, 64, 4, 16, new=(4, 300, 300, 33), ctx=(60, 2500, 2400, 700)), 0.0,
                                   SLOPES(32)),
}


@pytest.mark.parametrize("name", sorted(SHORT_TABLES))
def test_table_shorter_than_the_length(name):
    """Keys past a row's page table are left out and reported; the next row's pages are not read for them."""
    w = SHORT_TABLES[name]()
    att = _att(w)
    att.max_kv_len = max(att.max_kv_len, 200)
    from context_paged_attention_gb300 import binding as B

    att.workspace = torch.empty(B.workspace_bytes(att.desc, w.num_q_heads, w.num_tokens, att.max_kv_len),
                                dtype=torch.uint8, device="cuda")
    att.kv_len[0] = 64  # the first row's four pages, full
    for run in (att.run_step, att.run_step_fused):
        want = [x.clone() for x in run()]
        torch.cuda.synchronize()
        assert att.status() == 0
        att.kv_len[0] = 64 + 75
        got = [x.clone() for x in run()]
        torch.cuda.synchronize()
        assert att.status() == 2
        att.dev_status.zero_()
        att.kv_len[0] = 64
        n = int(w.qo_indptr[w.num_real_rows])
        top = float(want[0][:n].abs().max())
        # the split may differ with the lengths: two results of one definition
        torch.testing.assert_close(got[0][:n].float(), want[0][:n].float(), rtol=0, atol=2 ** -6 * top)
        torch.testing.assert_close(got[1][:n], want[1][:n], rtol=0, atol=2e-4 + 2 ** -19 * float(want[1][:n].abs().max()))


def test_partials_without_a_workspace():
    """The call with the library's own scratch takes 4-bit pools too, split stripes among them."""
    import ctypes

    from context_paged_attention_gb300 import binding as B

    lib = ctypes.CDLL(B.library_path())
    fn, vp, i32 = lib.cp_paged_attn_partial_noalloc, ctypes.c_void_p, ctypes.c_int32
    fn.argtypes = [ctypes.POINTER(B.PoolDesc), vp, vp, vp, i32, i32, i32, vp, vp, i32, vp, vp, ctypes.c_float, vp, vp,
                   vp, vp]
    for name in ("fp4_split", "fp4_mixed_g1_split"):
        w = STEPS[name]()
        att = _att(w)
        att.run_step()
        o, l_ = torch.full_like(att.o_parts[:w.P], 7.0), torch.full_like(att.lse_parts[:w.P], 7.0)
        st = fn(ctypes.byref(att.desc), att.pool_k.data_ptr(), att.pool_v.data_ptr(), att.q.data_ptr(), w.num_q_heads,
                w.num_rows, w.num_tokens, att.qo_indptr.data_ptr(), att.kv_len.data_ptr(), att.max_kv_len,
                att.page_indptr.data_ptr(), att.page_indices.data_ptr(), w.scale, o.data_ptr(), l_.data_ptr(),
                att.dev_status.data_ptr(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == 0 and att.status() == 0
        att.partial()
        torch.cuda.synchronize()
        assert torch.equal(o, att.o_parts[:w.P]) and torch.equal(l_, att.lse_parts[:w.P])


def test_extreme_scores():
    """Capped scores far past the cap on both sides stay +-cap, and equal weights follow."""
    w = W.scored(_decode(82, 4, 1, 64, 1, 16, [40, 200], qs=2.0 ** 20), 12.0)
    for wl in (w, F8(w)):
        # E4M3 kernels multiply queries as float16: keep them in its range
        wl = wl if wl.kv_dtype == "same" else dataclasses.replace(wl, q=W.scored(
            _decode(82, 4, 1, 64, 1, 16, [40, 200], qs=2.0 ** 12), 12.0).q)
        att = _att(wl)
        att.run_step()
        torch.cuda.synchronize()
        assert np.all(np.isfinite(f64(att.out)))
        check_step(wl, att, att.out, att.lse)


def test_workspace_contents_do_not_matter(step):
    w, att = step
    for run in (att.run_step, att.run_step_fused):
        a = [x.clone() for x in run()]
        for ws in (att.workspace, att._fused_ws):
            if ws is not None:
                ws.fill_(0xFF)
        b = run()
        torch.cuda.synchronize()
        assert att.status() == 0
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_calls_at_once():
    """Steps of different shapes on two streams, each with its own workspace."""
    atts = [_att(STEPS[n]()) for n in ("mixed_many", "fp4_split", "mixed_fp4", "both_e4m3")]
    want = [[x.clone() for x in att.run_step_fused()] for att in atts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in atts]
    for att in atts:
        att.out.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for att, s in zip(atts, streams):
            att.run_step_fused(s)
    torch.cuda.synchronize()
    for att, (o, l_) in zip(atts, want):
        assert att.status() == 0 and torch.equal(att.out, o) and torch.equal(att.lse, l_)


@pytest.mark.parametrize("name", ["mixed_many", "mixed_many_e4m3", "fp4_split", "mixed_fp4", "split"])
def test_replay_with_other_lengths(name):
    """Work is split by the lengths on the device: a captured step follows them."""
    w = STEPS[name]()
    att = _att(w)
    att.capture(fused=True)
    full = att.kv_len.clone()
    for lens in (full // 2, full * 0 + 1, full * 0, full):
        att.kv_len.copy_(torch.minimum(lens.clamp(min=1) if w.decode else lens, full))
        o, l_ = (x.clone() for x in att.replay())
        torch.cuda.synchronize()
        assert att.status() == 0
        a = [x.clone() for x in att.run_step_fused()]
        b = att.run_step()
        torch.cuda.synchronize()
        assert torch.equal(o, a[0]) and torch.equal(l_, a[1])
        n = int(w.qo_indptr[w.num_real_rows])
        # each path is within 2^-7 of the largest value's size of the definition
        torch.testing.assert_close(o[:n].float(), b[0][:n].float(), rtol=2 ** -6, atol=2 ** -6 * float(b[0][:n].abs().max()))


def test_other_device_is_refused(monkeypatch):
    from context_paged_attention_gb300 import binding as B

    atts = [_att(STEPS[n]()) for n in ("layer_plain", "fp4_g8", "cap_bf16", "mixed")]
    for att in atts:
        att.run_step()
        att.run_step_fused()
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream()
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    for att in atts:
        with pytest.raises(ValueError, match="current CUDA device"):
            att.run_step(stream)
        with pytest.raises(ValueError, match="current CUDA device"):
            att.run_step_fused(stream)


def test_other_stream_and_full_size_sample():
    """The full-size 4-bit decode batch on a side stream, sampled rows."""
    w = W.rotated(W.gqa_decode_fp4(batch=64), 128)
    att = _att(w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    att.run_step_fused(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert att.status() == 0 and bool(torch.isfinite(att.out.float()).all())
    check_step(w, att, att.out, att.lse, rows=[0, 31, 63])
