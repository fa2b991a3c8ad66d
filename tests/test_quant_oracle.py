"""Pins of the 8-bit cache's oracle (CPU), and the checks of arguments that need no GPU."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import lora_shared_kv_b200 as lrkv
import oracle
from oracle import kvq_oracle as kvq


def test_e4m3_numbers_are_torchs():
    bits = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(bits).view(torch.float8_e4m3fn).double().numpy()
    got = kvq.e4m3_from_bits(bits)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_e4m3_rounding_is_torchs_cast():
    x = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    x = x[x <= 448]
    want = x.float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kvq.nearest(x.numpy(), "e4m3"), want)
    assert np.array_equal(kvq.nearest(-x.numpy(), "e4m3"), -want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scale_is_the_smallest_that_holds_the_block(fmt):
    rng = np.random.default_rng(3)
    bits = rng.integers(1, 0x7F80, 4000).astype(np.uint16)
    for a in oracle.bf16_bits_to_f64(bits):
        s = Fraction(kvq.scale_for(float(a), fmt))
        top = Fraction(int(kvq.TOP[fmt]))
        assert Fraction(a) <= top * s
        if s == Fraction(kvq.SCALE_MIN):
            continue
        if fmt == "e4m3":
            assert s.numerator & (s.numerator - 1) == 0 and s.denominator & (s.denominator - 1) == 0
            below = s / 2
        else:
            f = np.float64(float(s)).astype(np.float32).view(np.uint32)
            assert Fraction(float(s)) == s and f & 0xFFFF == 0  # a bf16 number
            below = Fraction(float((f - np.uint32(0x10000)).view(np.float32)))
        assert Fraction(a) > top * below


def test_int8_rounding_on_rationals():
    rng = np.random.default_rng(5)
    for _ in range(2000):
        s = float(oracle.bf16_bits_to_f64(np.array([rng.integers(0x3000, 0x4800)], dtype=np.uint16))[0])
        n = int(rng.integers(-120, 121))
        x = float(np.float32((n + rng.choice([0.0, 0.5, 0.25, 0.4999])) * s))
        want = round(Fraction(x) / Fraction(s))  # Python rounds half to even
        assert kvq.nearest(np.array([x / s]), "int8")[0] == max(-127, min(127, want))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_errors_are_half_a_step(fmt):
    rng = np.random.default_rng(7)
    x = oracle.bf16_bits_to_f64(oracle.f32_to_bf16_bits_rne((rng.normal(size=(150, 2, 8)) * np.exp(rng.normal(
        size=(150, 1, 1)))).astype(np.float32)))
    codes, scales = np.zeros((2, 192, 8)), np.zeros((2, 3))
    kvq.write(codes, scales, x, 0, fmt)
    y = kvq.values(codes, scales)[:, :150].transpose(1, 0, 2)
    s = np.repeat(scales, 64, axis=1)[:, :150].T[..., None]
    half = s / 2 if fmt == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10)
    assert np.all(np.abs(y - x) <= half)


def test_a_growing_e4m3_scale_keeps_the_block():
    # rows whose codes stay normal numbers after the scale grows by 2^6 come through unchanged
    x = np.full((10, 1, 4), 3.25)
    codes, scales = np.zeros((1, 64, 4)), np.zeros((1, 1))
    kvq.write(codes, scales, x, 0, "e4m3")
    before = kvq.values(codes, scales)[:, :10].copy()
    kvq.write(codes, scales, np.full((1, 1, 4), 208.0), 10, "e4m3")
    assert scales[0, 0] == 2.0 ** -1 and np.array_equal(kvq.values(codes, scales)[:, :10], before)


def test_append_in_pieces_of_e4m3_is_one_write():
    # power-of-two scales: without values that fall below the smallest step, how a block is filled plays no part
    rng = np.random.default_rng(9)
    x = np.sign(rng.normal(size=(130, 2, 4))) * (1 + rng.random((130, 2, 4)) * 30)
    a, sa = np.zeros((2, 192, 4)), np.zeros((2, 3))
    b, sb = np.zeros((2, 192, 4)), np.zeros((2, 3))
    kvq.write(a, sa, x, 0, "e4m3")
    at = 0
    for n in (1, 7, 60, 1, 61):
        kvq.write(b, sb, x[at:at + n], at, "e4m3")
        at += n
    assert np.array_equal(sa, sb) and np.array_equal(a, b)


def test_decode_with_bound_is_the_oracles_decode():
    rng = np.random.default_rng(11)
    S, N, Hq, Hkv, d, r, L = 2, 3, 4, 2, 8, 4, 70
    q, k, v = rng.normal(size=(S, N, Hq, d)), rng.normal(size=(S, Hkv, L, d)), rng.normal(size=(S, Hkv, L, d))
    b = rng.normal(size=(N, r, Hkv * d))
    offs, sl = np.array([[0, 20, 90], [5, 69, 70]]), np.array([70, 33])
    for mode in (0, 1):
        u = rng.normal(size=(S, N if mode == 0 else 1, L, r))
        out, a_v, a_z, _ = kvq.decode_with_bound(q, k, v, u, b, offs, sl, mode)
        assert np.allclose(out, oracle.decode(q, k, v, u, b, offs, sl, mode), rtol=1e-12, atol=1e-13)
        assert np.all(np.abs(out) <= a_v + a_z + 1e-12)


# ---------------------------------------------------------------------------
# refusals, before anything touches a device
# ---------------------------------------------------------------------------

FAKE = 0x10000  # never dereferenced


def _problem(**kw):
    a = dict(S=2, N=3, Hq=12, Hkv=2, d=128, r=16, mode=0)
    a.update(kw)
    return lrkv.make_problem(a["S"], a["N"], a["Hq"], a["Hkv"], a["d"], a["r"], a["mode"])


def _qkv(**kw):
    v = lrkv.QKVView(FAKE, FAKE, FAKE, FAKE, 2 * 8192 * 128, 8192 * 128, 128, 256, 128)
    for name, x in kw.items():
        setattr(v, name, x)
    return v


def _paged(**kw):
    a = dict(page_table=FAKE, page_table_stride=128, stride_page=2 * 64 * 128, scale_stride_page=2, page_size=64,
             num_pages=300, stride_head=64 * 128, scale_stride_head=1)
    a.update(kw)
    return _qkv(**a)


def _kv(**kw):
    v = lrkv.KVView(FAKE, FAKE, 2 * 8192 * 128, 8192 * 128, 128, None, 0, 0, 0, 0)
    for name, x in kw.items():
        setattr(v, name, x)
    return v


BAD_VIEWS = [
    (_qkv(k=None), 1), (_qkv(v=None), 1), (_qkv(k_scale=None), 1), (_qkv(v_scale=None), 1), (_qkv(format=2), 1),
    (_qkv(k=FAKE + 8), 3), (_qkv(v_scale=FAKE + 2), 3), (_qkv(stride_token=64), 1), (_qkv(stride_token=136), 3),
    (_qkv(stride_head=0), 1), (_qkv(stride_head=8), 3), (_qkv(scale_stride_head=0), 1), (_qkv(stride_session=0), 3),
    (_qkv(stride_session=8), 3), (_qkv(scale_stride_session=0), 1), (_paged(page_size=32), 2),
    (_paged(num_pages=0), 1), (_paged(stride_page=24), 1), (_paged(page_table_stride=0), 1),
    (_paged(scale_stride_page=0), 1),
]


def _quantize(prob=None, src=None, T=4, dst=None, rows=8192, first=FAKE, ws=FAKE, nbytes=256):
    L = lrkv.lib()
    return L.lrkv_quantize_kv(ctypes.byref(prob or _problem()), ctypes.byref(src or _kv()), T,
                              ctypes.byref(dst or _qkv()), rows, first, None, ws, nbytes, None)


def _dequantize(prob=None, src=None, T=4, dst=None, rows=8192, first=FAKE, ws=FAKE, nbytes=256):
    L = lrkv.lib()
    return L.lrkv_dequantize_kv(ctypes.byref(prob or _problem()), ctypes.byref(src or _qkv()), rows, T,
                                ctypes.byref(dst or _kv()), first, None, ws, nbytes, None)


def _decode(prob=None, kv=None, q=FAKE, max_len=8192, nbytes=1 << 30, u_rows=8192, dtype=0, ws=FAKE):
    L = lrkv.lib()
    uv = lrkv.UView(FAKE, 3 * 8192 * 16, 8192 * 16, 16, u_rows)
    return L.lrkv_attn_decode_quant(ctypes.byref(prob or _problem()), q, ctypes.byref(kv or _qkv()), FAKE, max_len,
                                    ctypes.byref(uv), FAKE, None, FAKE, dtype, ws, nbytes, None)


@pytest.mark.parametrize("view,status", BAD_VIEWS, ids=range(len(BAD_VIEWS)))
def test_bad_views_are_refused(view, status):
    assert _quantize(dst=view) == status
    assert _dequantize(src=view) == status
    assert _decode(kv=view) == status


def test_bad_arguments_of_write_and_read():
    for call in (_quantize, _dequantize):
        assert call(prob=_problem(d=96)) == 2
        assert call(T=-1) == 1
        assert call(rows=-1) == 1
        assert call(T=9000, first=None) == 1     # more rows than the cache holds
        assert call(T=9000) == 1
        assert call(rows=(1 << 30) + 1) == 2
        assert call(ws=None) == 1
        assert call(ws=FAKE + 4) == 3
        assert call(nbytes=255) == 4
    assert _quantize(src=_kv(k=None)) == 1 and _dequantize(dst=_kv(v=FAKE + 2)) == 3
    assert _quantize(dst=_paged(page_table_stride=64)) == 1   # 8192 rows need 128 pages
    assert _dequantize(src=_paged(page_table_stride=64)) == 1
    short = _kv(page_table=FAKE, page_table_stride=1, stride_page=1 << 15, page_size=64, num_pages=4)
    assert _quantize(src=short, T=65) == 1 and _dequantize(dst=short, T=65) == 1
    assert _quantize(T=0) == 0 and _dequantize(T=0) == 0      # nothing to do, nothing launched


def test_bad_arguments_of_decode():
    assert _decode(prob=_problem(d=96)) == 2 and _decode(prob=_problem(r=12)) == 2
    assert _decode(prob=_problem(N=17)) == 2
    assert _decode(q=None) == 1 and _decode(q=FAKE + 2) == 3 and _decode(ws=FAKE + 8) == 3
    assert _decode(max_len=-1) == 1 and _decode(dtype=2) == 1
    assert _decode(max_len=8193) == 1                          # past the U capacity
    assert _decode(kv=_paged(page_table_stride=127)) == 1
    assert lrkv.lib().lrkv_decode_quant_workspace_bytes(ctypes.byref(_problem(d=96)), 100) == 0
    assert lrkv.lib().lrkv_decode_quant_workspace_bytes(ctypes.byref(_problem()), -1) == 0


def test_workspace_does_not_grow_with_the_context():
    # two partial records per CTA, however long the sessions
    a = lrkv.lrkv_decode_quant_workspace_bytes(_problem(), 8192)
    assert a == lrkv.lrkv_decode_quant_workspace_bytes(_problem(), 65536)
    items = 2 * 2
    assert a == 256 + -(-items * 4 // 256) * 256 + 2 * 148 * 24 * (128 + 16 + 2) * 4  # 18 rows take a 24-row record


def test_binding_refuses_before_the_library():
    k8 = torch.zeros((1, 2, 64, 128), dtype=torch.int8)
    sc = torch.ones((1, 2, 1))
    with pytest.raises(ValueError, match="CUDA tensor"):
        lrkv.kv_view_quant_dense(k8, k8, sc, sc)
    with pytest.raises(ValueError, match="float8_e4m3fn or int8"):
        lrkv.kv_view_quant_dense(k8.half(), k8.half(), sc, sc)
    with pytest.raises(ValueError, match="float8_e4m3fn or int8"):
        lrkv.kv_view_quant_dense(k8, k8.float().to(torch.float8_e4m3fn), sc, sc)
    with pytest.raises(ValueError, match="fp32"):
        lrkv.kv_view_quant_dense(k8, k8, sc.double(), sc.double())
    with pytest.raises(ValueError, match="same strides"):
        lrkv.kv_view_quant_dense(k8, k8.transpose(1, 2).contiguous().transpose(1, 2), sc, sc)
