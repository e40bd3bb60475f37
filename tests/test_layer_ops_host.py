"""Rotated appends, 4-bit pools and modified scores without a GPU: the oracle's
definitions against closed forms and library routines, the host-side refusals
of the C calls (each fails before anything is launched), and the binding's
argument checks."""

import ctypes
import dataclasses
import math

import numpy as np
import pytest
import torch

import oracle
from context_paged_attention_gb300 import binding as B
from context_paged_attention_gb300 import build_lib
from context_paged_attention_gb300 import workloads as W
from context_paged_attention_gb300.step import desc_for, rope_table

FAKE = 0x10000  # never dereferenced: these calls fail host validation first


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return B.load_library()


# ---------------------------------------------------------------- the oracle

def test_e2m1_values_and_rounding():
    mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert [oracle.e2m1_value(c) for c in range(16)] == mags + [-m for m in mags]
    # midpoints go to the even code, everything past 6 to 6
    for lo in range(7):
        mid = (mags[lo] + mags[lo + 1]) / 2
        assert oracle.e2m1_encode(mid) == (lo if lo % 2 == 0 else lo + 1)
        assert oracle.e2m1_encode(np.nextafter(mid, 0)) == lo
        assert oracle.e2m1_encode(np.nextafter(mid, 9)) == lo + 1
    assert oracle.e2m1_encode(1e9) == 7 and oracle.e2m1_encode(-np.inf) == 15


def test_fp4_rows_closed_forms():
    # a block of multiples of its own scale is stored exactly
    x = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -1.5, -2, -3, -4, -6, 0], np.float32)
    codes, s = oracle.fp4_quantize(x[None] * 0.25, 0.125)
    assert oracle.e4m3_value(s[0, 0]) == 2.0
    assert np.array_equal(oracle.fp4_dequantize(codes, s, 0.125)[0], x.astype(np.float64) * 0.25)
    # zeros, a block below the smallest scale, NaN, infinity
    z = np.zeros((4, 16), np.float32)
    z[1] = 1e-4
    z[2, 3] = np.nan
    z[3, 5], z[3, 6] = np.inf, 1000.0
    codes, s = oracle.fp4_quantize(z, 1.0)
    d = oracle.fp4_dequantize(codes, s, 1.0)
    assert np.all(d[0] == 0) and np.all(d[1] == 0) and np.all(np.isnan(d[2]))
    assert d[3, 5] == 448 * 6 and d[3, 6] == 448 * 2
    assert np.array_equal(oracle.fp4_pack(np.arange(16)[None] % 16)[0],
                          [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE])


def test_fp4_error_bound():
    """|stored - x| <= half an E2M1 step at the block's scale: codes go up to 6,
    the scale is off by at most 2^-4 of max / 6, so a value is off by at most
    (1/6 + 1/16) of the block's largest (a step of 2 near 6 is a third of it)."""
    x = np.random.default_rng(0).standard_normal((200, 128)).astype(np.float32)
    codes, s = oracle.fp4_quantize(x, 0.0021)
    err = np.abs(oracle.fp4_dequantize(codes, s, 0.0021) - x).reshape(-1, 16)
    assert np.all(err <= (1 / 6 + 1 / 16) * np.abs(x).reshape(-1, 16).max(1, keepdims=True))
    assert np.any(err > 0.1 * np.abs(x).reshape(-1, 16).max(1, keepdims=True))


def test_scale_rounding_matches_torch_e4m3():
    x = np.abs(np.random.default_rng(1).standard_normal((4000, 16))).astype(np.float32) * 2500
    _, s = oracle.fp4_quantize(x, 1.0)
    q = torch.tensor(x.max(1) / np.float32(6)).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(s[:, 0], q)


def test_rotation_closed_forms():
    x = np.random.default_rng(2).standard_normal((3, 2, 8))
    tab = rope_table(50, 4)
    for style in (oracle.ROPE_HALVES, oracle.ROPE_PAIRS):
        y = oracle.rotate(x, [0, 7, -1], tab, 2, style)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[2], x[2])  # position 0 and padding: unchanged
        assert np.array_equal(y[..., :2], x[..., :2]) and np.array_equal(y[..., 6:], x[..., 6:])
        assert np.allclose((y[1, :, 2:6] ** 2).sum(-1), (x[1, :, 2:6] ** 2).sum(-1))  # a rotation
    # the product of two rows depends on the distance only
    a, b = np.random.default_rng(3).standard_normal((2, 1, 1, 64))
    tab = rope_table(200, 64)
    d = [float((oracle.rotate(a, [n + 9], tab, 0, 0) * oracle.rotate(b, [n], tab, 0, 0)).sum()) for n in (0, 40, 190)]
    assert max(d) - min(d) < 1e-5  # the table is float32


def test_modified_attention_against_logsumexp():
    from scipy.special import logsumexp, softmax
    rng = np.random.default_rng(4)
    q, K, V = rng.standard_normal((4, 16)), rng.standard_normal((9, 2, 16)), rng.standard_normal((9, 2, 16))
    slopes = np.array([0.5, 0.25, -0.1, 0.0])
    O, L, A, Bd = oracle.modified_attention(q, K, V, 0.7, 12, np.arange(9), 2.5, slopes)
    for h in range(4):
        s = 2.5 * np.tanh(0.7 * K[:, h // 2] @ q[h] / 2.5) + slopes[h] * (np.arange(9) - 12)
        assert np.allclose(O[h], softmax(s) @ V[:, h // 2]) and np.isclose(L[h], logsumexp(s))
        assert np.allclose(A[h], softmax(s) @ np.abs(V[:, h // 2])) and np.all(Bd[h] >= A[h] - 1e-12)
    O, L = oracle.attention(q, K, V, 0.7)
    O2, L2, _, _ = oracle.modified_attention(q, K, V, 0.7, 0, np.arange(9))
    assert np.allclose(O, O2) and np.allclose(L, L2)
    O0, L0, _, _ = oracle.modified_attention(q, K[:0], V[:0], 0.7, 0, [], 3.0, slopes)
    assert np.all(O0 == 0) and np.all(L0 == -np.inf)


# ---------------------------------------------------------------- refusals of the C calls

def _desc(**kw):
    d = dict(P=4, page_size=16, num_pages=10, num_kv_heads=8, head_dim=128, head_dim_v=128, dtype=B.DTYPE_BF16)
    d.update(kw)
    return B.PoolDesc(**d)


def test_fp4_descriptor_checks(lib):
    fp4 = dict(kv_dtype=B.DTYPE_FP4_E2M1, k_descale=0.002, v_descale=0.002)
    assert lib.cpattn_pool_bytes(ctypes.byref(_desc(**fp4)), 0) == 4 * 10 * 8 * 4 * (64 + 8)
    assert lib.cp_paged_attn_workspace_bytes(ctypes.byref(_desc(**fp4)), 32, 64, 8192) > 0
    assert lib.cpattn_pool_bytes(ctypes.byref(_desc(dtype=B.DTYPE_FP32, **fp4)), 0) == 0
    assert lib.cpattn_pool_bytes(ctypes.byref(_desc(head_dim=80, head_dim_v=80, **fp4)), 0) == 0  # not blocks of 32
    for s in (0.0, -1.0, math.nan, math.inf):
        assert lib.cpattn_pool_bytes(ctypes.byref(_desc(kv_dtype=3, k_descale=s, v_descale=1.0)), 0) == 0
    mla = _desc(num_kv_heads=1, head_dim=576, head_dim_v=512, page_size=64, **fp4)
    assert lib.cp_paged_attn_partial(ctypes.byref(mla), FAKE, FAKE, FAKE, 128, 1, 1, None, FAKE, 100, FAKE, FAKE, 0.1,
                                     FAKE, FAKE, FAKE, 1 << 30, None, None) == -3
    # rows past 32-bit indices
    huge = _desc(num_pages=1 << 26, **fp4)
    assert lib.cp_paged_attn_partial(ctypes.byref(huge), FAKE, FAKE, FAKE, 32, 2, 2, None, FAKE, 100, FAKE, FAKE, 0.1,
                                     FAKE, FAKE, FAKE, 1 << 30, None, None) == -3
    # head widths and group sizes without a kernel
    for kw, hq in ((dict(head_dim=96, head_dim_v=96), 32), (dict(), 24), (dict(num_kv_heads=1), 32)):
        assert lib.cp_paged_attn_partial(ctypes.byref(_desc(**kw, **fp4)), FAKE, FAKE, FAKE, hq, 1, 1, None, FAKE, 100,
                                         FAKE, FAKE, 0.1, FAKE, FAKE, FAKE, 1 << 30, None, None) == -3


def _rope_args(d, q=FAKE, k=FAKE, v=FAKE, hq=32, rows=1, tokens=1, cs=FAKE, table=100, begin=0, dim=128, style=0,
               q_out=FAKE, k_out=None, pos=FAKE, pool_v=FAKE):
    return (ctypes.byref(d), FAKE, pool_v, q, k, v, hq, pos, FAKE, rows, tokens, FAKE, FAKE, cs, table, begin, dim, style,
            q_out, k_out, None, None)


def test_rope_write_refusals(lib):
    f, d = lib.cp_rope_kv_write, _desc()
    assert f(*_rope_args(d, tokens=0)) == 0  # nothing to do
    for kw in (dict(style=2), dict(style=-1), dict(dim=0), dict(dim=7), dict(dim=130), dict(begin=-1),
               dict(begin=2, dim=128), dict(begin=2147483647, dim=128), dict(table=0), dict(q=None), dict(q_out=None),
               dict(hq=0), dict(k=None), dict(v=None), dict(cs=None), dict(pos=None), dict(rows=0), dict(tokens=-1),
               dict(pool_v=None)):
        assert f(*_rope_args(d, **kw)) == -1, kw
    for kw in (dict(q=FAKE + 2), dict(q_out=FAKE + 8), dict(k_out=FAKE + 4), dict(cs=FAKE + 4), dict(k=FAKE + 2)):
        assert f(*_rope_args(d, **kw)) == -4, kw
    assert f(*_rope_args(_desc(P=3))) == -2
    mla = _desc(num_kv_heads=1, head_dim=576, head_dim_v=512, page_size=64)
    assert f(*_rope_args(mla, begin=512, dim=64)) == -1  # MLA takes no values
    assert f(*_rope_args(_desc(head_dim=4096, head_dim_v=4096))) == -3


def test_score_mod_refusals(lib):
    d = _desc()

    def fused(mod, desc=d, hq=32):
        return lib.cp_paged_attn_fused_mod(ctypes.byref(desc), FAKE, FAKE, FAKE, hq, 1, 1, None, FAKE, 100, FAKE, FAKE,
                                           None, 0.1, None, None, 0, FAKE, None, mod, FAKE, 0, None, None)

    def own(mod, mla=False):
        return lib.own_token_attn_mod(FAKE, FAKE, None if mla else FAKE, 32, 1 if mla else 8, 576 if mla else 128,
                                      512 if mla else 128, 0, FAKE, 4, 4, 0, 8, 0.1, mod, FAKE, FAKE, None)

    for cap in (-1.0, math.nan, math.inf, 1e-9, 1e35):
        m = B.ScoreMod(cap, None, None)
        assert fused(m) == -1 and own(m) == -1
        assert lib.cp_paged_attn_partial_mod(ctypes.byref(d), FAKE, FAKE, FAKE, 32, 1, 1, None, FAKE, 100, FAKE, FAKE,
                                             0.1, FAKE, FAKE, 0, None, m, FAKE, 0, None, None) == -1
    # accepted, then stopped by the empty workspace (no launch); no tokens: nothing to do
    for m in (None, B.ScoreMod(0.0, None, None), B.ScoreMod(30.0, FAKE, FAKE)):
        assert fused(m) == -5 and own(m) == 0
    mla = _desc(num_kv_heads=1, head_dim=576, head_dim_v=512, page_size=64)
    m = B.ScoreMod(30.0, None, None)
    assert lib.cp_paged_attn_partial_mod(ctypes.byref(mla), FAKE, None, FAKE, 128, 1, 1, None, FAKE, 100, FAKE, FAKE,
                                         0.1, FAKE, FAKE, 0, None, m, FAKE, 0, None, None) == -3
    assert own(m, mla=True) == -3


def test_longest_rows(lib):
    """Lengths that 32-bit rounding up would wrap are refused for 4-bit pools and modified scores."""
    d, f4, m = _desc(), _desc(kv_dtype=B.DTYPE_FP4_E2M1, k_descale=0.002, v_descale=0.002), B.ScoreMod(30.0, None, None)
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        for desc, mod in ((d, m), (f4, None)):
            assert lib.cp_paged_attn_fused_mod(ctypes.byref(desc), FAKE, FAKE, FAKE, 32, 1, 1, None, FAKE, n, FAKE, FAKE,
                                               None, 0.1, None, None, 0, FAKE, None, mod, FAKE, 1 << 40, None, None) == -3
            assert lib.cp_paged_attn_partial_mod(ctypes.byref(desc), FAKE, FAKE, FAKE, 32, 1, 1, None, FAKE, n, FAKE,
                                                 FAKE, 0.1, FAKE, FAKE, 0, None, mod, FAKE, 1 << 40, None, None) == -3
        assert lib.cp_paged_attn_fused_workspace_bytes(ctypes.byref(f4), 32, 1, n) == 0
        assert lib.cp_paged_attn_workspace_bytes(ctypes.byref(f4), 32, 1, n) == 0
    # multi-token rows whose pool rows pass 31 bits
    e4 = _desc(kv_dtype=B.DTYPE_FP8_E4M3, k_descale=0.01, v_descale=0.01, num_pages=1 << 24)
    assert lib.cp_paged_attn_fused_mod(ctypes.byref(e4), FAKE, FAKE, FAKE, 32, 1, 2, FAKE, FAKE, 100, FAKE, FAKE, None, 0.1,
                                       None, None, 0, FAKE, None, m, FAKE, 1 << 40, None, None) == -3


# ---------------------------------------------------------------- binding and workloads

def test_binding_checks_shapes(lib):
    d = _desc()
    x = torch.zeros(2, 32, 128, dtype=torch.bfloat16)
    k = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    tab = torch.zeros(4, 128)
    call = lambda q=x, kn=k, v=k, t=tab, qo=x: B.cp_rope_kv_write(d, k, k, q, kn, v, i, i, i, i, t, qo)  # noqa: E731
    for kw, err in ((dict(t=tab.double()), TypeError), (dict(t=tab[0]), TypeError), (dict(q=x.float()), TypeError),
                    (dict(kn=k[:1]), ValueError), (dict(v=k[..., :64]), ValueError), (dict(qo=x[:, :8]), ValueError),
                    (dict(), ValueError)):  # the last: CPU tensors
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(TypeError):
        B.score_mod(1.0, torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        B.score_mod(1.0, torch.zeros(4))
    m = B.ScoreMod(1.0, None, None)
    m.tensors = (torch.zeros(4), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        B._mod(m, 5, 3)
    with pytest.raises(ValueError):
        B._mod(m, 4, 2)


def test_workload_variants():
    w = W.gqa_decode(seed=3, batch=2, len_lo=5, len_hi=40)
    f = W.fp4_pool(w, 0.002, 0.003)
    assert f.kv_bytes_read() * 32 == w.kv_bytes_read() * 9
    d = desc_for(f)
    assert d.fp4 and d.pool_shape() == (4 * w.num_pages * 8 * 4 * 72,)
    codes, scales = d.fp4_views(torch.arange(d.pool_shape()[0]) % 251)
    assert codes.shape == (4, w.num_pages, 8, 4, 64) and scales.shape == (4, w.num_pages, 8, 4, 8)
    assert codes.flatten()[-1] + 1 == scales.flatten()[0] or scales.flatten()[0] == 0
    for bad in (dict(rot_dim=3), dict(rot_dim=130), dict(rot_dim=64, rot_begin=65)):
        with pytest.raises(ValueError):
            W.rotated(w, **bad)
    with pytest.raises(ValueError):
        W.scored(w, slopes=np.ones(3))
    with pytest.raises(ValueError):
        W.fp4_pool(W.tiny_fp32(), 1.0, 1.0)
    assert W.scored(w, 30.0, np.ones(32)).slopes.dtype == np.float32
    assert dataclasses.replace(w).rot_dim == 0
