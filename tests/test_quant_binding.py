"""The binding of the 8-bit cache's calls refuses, before any call into the library, views that do not hold what
the kernels would read.  Runs without a GPU: host tensors stand for device ones, and the library is replaced by an
object that fails the test if anything reaches it."""

import pytest
import torch

import lora_shared_kv_b200 as lrkv

S, N, G, Hkv, d, r, L = 2, 3, 6, 2, 128, 16, 256
Hq = G * Hkv


class _NoLibrary:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was called although the arguments were invalid")


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(lrkv, "_lib", _NoLibrary())
    monkeypatch.setattr(lrkv, "_on_device", lambda **tensors: None)  # host tensors pass for the current device's
    monkeypatch.setattr(lrkv, "_on_current", lambda *tensors: 0)


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _kv8():
    codes = torch.zeros((S, Hkv, L, d), dtype=torch.int8)
    return lrkv.kv_view_quant_dense(codes, codes.clone(), torch.ones(S, Hkv, L // 64), torch.ones(S, Hkv, L // 64))


def _decode(u, mode=lrkv.BASE_SHARED, max_seq_len=L, kv=None):
    prob = lrkv.make_problem(S, N, Hq, Hkv, d, r, mode)
    lrkv.lrkv_attn_decode_quant(prob, _bf16(S, N, Hq, d), kv or _kv8(), _i32(S), max_seq_len, u,
                                _bf16(N, r, Hkv * d), None, _bf16(S, N, Hq, d), torch.zeros(1 << 20, dtype=torch.uint8),
                                stream=0)


U_TOO_SMALL = {
    "one agent's U for three": (S, 1, L, r),
    "a U short of an agent": (S, N - 1, L, r),
    "fewer sessions": (S - 1, N, L, r),
    "fewer rows": (S, N, L - 1, r),
    "a smaller rank": (S, N, L, r // 2),
    "a larger rank": (S, N, L, 2 * r),
}


@pytest.mark.parametrize("shape", U_TOO_SMALL.values(), ids=U_TOO_SMALL)
def test_a_u_that_does_not_hold_the_problem_is_refused(shape):
    for u in (_bf16(*shape), lrkv.u_view(_bf16(*shape))):
        with pytest.raises(ValueError, match="U view holds"):
            _decode(u)


def test_a_shared_u_needs_one_slot_only():
    with pytest.raises(AssertionError, match="lrkv_attn_decode_quant"):  # reaches the library
        _decode(_bf16(S, 1, L, r), lrkv.BASE_LR_SHARED)
    with pytest.raises(AssertionError, match="lrkv_attn_decode_quant"):
        _decode(_bf16(S, N, L, r))
    with pytest.raises(ValueError, match="U view holds"):
        _decode(_bf16(S - 1, 1, L, r), lrkv.BASE_LR_SHARED)


def test_a_us_device_is_checked(monkeypatch):
    seen = []
    monkeypatch.setattr(lrkv, "_on_current", lambda *tensors: seen.extend(tensors) or 0)
    u = _bf16(S, N, L, r)
    with pytest.raises(AssertionError, match="lrkv_attn_decode_quant"):
        _decode(lrkv.u_view(u))
    assert any(t is u for t in seen)


# ---------------------------------------------------------------------------
# bf16 views whose K and V differ
# ---------------------------------------------------------------------------

def _write(src, T, dst=None):
    prob = lrkv.make_problem(S, N, Hq, Hkv, d, r)
    lrkv.lrkv_quantize_kv(prob, src, T, dst or _kv8(), L, None, None, torch.zeros(256, dtype=torch.uint8), stream=0)


def _read(dst, T):
    prob = lrkv.make_problem(S, N, Hq, Hkv, d, r)
    lrkv.lrkv_dequantize_kv(prob, _kv8(), L, T, dst, None, None, torch.zeros(256, dtype=torch.uint8), stream=0)


V_TOO_SMALL = {"sessions": (slice(0, S - 1),), "heads": (slice(None), slice(0, Hkv - 1)),
               "rows": (slice(None), slice(None), slice(0, 99))}


@pytest.mark.parametrize("cut", V_TOO_SMALL.values(), ids=V_TOO_SMALL)
def test_a_dense_view_holds_what_both_of_its_tensors_hold(cut):
    k, v = _bf16(S, Hkv, 128, d), _bf16(S, Hkv, 128, d)
    for view in (lrkv.kv_view_dense(k, v[cut]), lrkv.kv_view_dense(k[cut], v)):
        for call in (_write, _read):
            with pytest.raises(ValueError, match="bf16 view holds"):
                call(view, 100)
    with pytest.raises(AssertionError, match="lrkv_quantize_kv"):
        _write(lrkv.kv_view_dense(k, v[:, :, :100]), 100)


def test_a_paged_view_holds_what_both_of_its_tensors_hold():
    k, v, table = _bf16(9, Hkv, 64, d), _bf16(9, Hkv, 64, d), _i32(S, 2)
    assert lrkv.kv_view_paged(k, v[:5], table).num_pages == 5  # the kernels flag page ids from there on
    assert lrkv.kv_view_paged(k[:4], v, table).num_pages == 4
    for call in (_write, _read):
        with pytest.raises(ValueError, match="bf16 view holds"):
            call(lrkv.kv_view_paged(k, v[:, :1], table), 100)
    with pytest.raises(ValueError, match="same page size"):
        lrkv.kv_view_paged(k, v[:, :, :32], table)


# ---------------------------------------------------------------------------
# views built by hand
# ---------------------------------------------------------------------------

def test_views_without_their_tensors_are_refused_with_a_message():
    kv = lrkv.KVView(0x1000, 0x1000, Hkv * L * d, L * d, d, None, 0, 0, 0, 0)
    kv8 = lrkv.QKVView(0x1000, 0x1000, 0x1000, 0x1000, Hkv * L * d, L * d, d, 8, 4)
    uv = lrkv.UView(0x1000, N * L * r, L * r, r, L)
    held = lrkv.kv_view_dense(_bf16(S, Hkv, 8, d), _bf16(S, Hkv, 8, d))
    for call in (lambda: _write(kv, 8), lambda: _read(kv, 8)):
        with pytest.raises(TypeError, match="kv_view_dense or kv_view_paged"):
            call()
    for call in (lambda: _write(held, 8, dst=kv8), lambda: _decode(_bf16(S, N, L, r), kv=kv8)):
        with pytest.raises(TypeError, match="kv_view_quant_dense or kv_view_quant_paged"):
            call()
    with pytest.raises(TypeError, match="u_view"):
        _decode(uv)
