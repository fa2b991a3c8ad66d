"""Decode over an 8-bit cache where scales are zero, tiny or far apart.

Bounds are those of test_gpu_quant, with what these cases add:

* A row's weights are relative to its largest; one below 2^-126 of it may count as zero
  (fp32's smallest normal number): |err| <= ... + 2^-126 sum_t |v|.
* Exponents are off by at most 128 * 2^-24 * sum |q k| scale, twice that where the tensor
  cores truncate, and again for the denominator: `weight` * 2^-12 with
  weight = 4 * 128 * 2^-12 * (largest score), 12 for scores up to 96.
"""

import numpy as np
import pytest
import torch

import lora_shared_kv_b200 as lrkv
from oracle import kvq_oracle as kvq
from test_gpu_quant import DEV, DecodeCase, _i32, _tokens

pytestmark = pytest.mark.gpu

FORMATS = ["e4m3", "int8"]
ROWS = [(2, 4), (2, 8), (3, 8), (4, 8), (1, 1)]  # agents, queries per KV head: 8, 16, 24, 2 x 16 rows and one


def _check(c, out, what, weight=1.0, floor=2.0 ** -33):
    ref, a_v, a_z, top = c.reference()
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got)), what
    v = np.nan_to_num(kvq.values(*c.cache.logical("v")), nan=0.0)
    lost = np.zeros_like(ref)
    for s, n in enumerate(c.lens):
        lost[s] = np.repeat(np.abs(v[s, :, :n]).sum(axis=1), c.G, axis=0)
    bound = (2.0 ** -11 * a_v + 2.0 ** -8 * a_z + weight * 2.0 ** -12 * (a_v + a_z) + floor * top
             + 2.0 ** -126 * lost)
    worst = np.max(np.abs(got - ref) / np.maximum(bound, 1e-300))
    assert worst <= 1.0, (what, worst)


# ---------------------------------------------------------------------------
# key scales that are zero or that the query's size takes below fp32
# ---------------------------------------------------------------------------

TAILS = [[148, 114], [129, 65], [1, 30], [160, 97]]  # the last blocks hold 20, 50; 1, 1; 1, 30; 32, 33 keys


@pytest.mark.parametrize("rows", ROWS, ids=str)
@pytest.mark.parametrize("fmt", FORMATS)
def test_zero_key_scale_in_a_partial_last_block(fmt, rows):
    N, G = rows
    for lens in TAILS:
        c = DecodeCase(("zk", fmt, rows, lens), fmt, 2, N, G, 2, 128, 16, 192, 0, [0, 40, 100, 7] * 2 if N == 4 else
                       [0, 40, 100][:N] * 2, lens)
        for s, n in enumerate(lens):
            c.cache.ks[s, :, (n - 1) // 64] = 0
        _check(c, c.run(), lens)


@pytest.mark.parametrize("rows", ROWS, ids=str)
@pytest.mark.parametrize("fmt", FORMATS)
def test_zero_keys_as_written_and_tiny_queries(fmt, rows):
    N, G = rows
    for lens in TAILS:
        c = DecodeCase(("tk", fmt, rows, lens), fmt, 2, N, G, 2, 64, 8, 192, 1, [0, 40, 100, 7] * 2 if N == 4 else
                       [0, 40, 100][:N] * 2, lens, paged=True, q_std=2.0 ** -40)
        first = [(n - 1) // 64 * 64 for n in lens]
        v = _tokens(("tk v", lens), 2, 64, 2, 64)
        c.cache.write(torch.zeros_like(v), v, 64, _i32(first), _i32([n - f for n, f in zip(lens, first)]))
        for s, n in enumerate(lens):
            assert (c.cache.logical("k")[1][s, :, (n - 1) // 64] == 2.0 ** -100).all()
        _check(c, c.run(), lens)


# ---------------------------------------------------------------------------
# value scales that are zero or far from those of a row's largest scores
# ---------------------------------------------------------------------------

def _sink(c, at, gap):
    """Give every row of c one key, `at`, whose score lies `gap` above the others' (which are all zero)."""
    S, L, H, d = c.cache.S, c.cache.rows, c.cache.Hkv, c.cache.d
    c.q[:] = 1.0
    k = torch.zeros((S, L, H, d), dtype=torch.bfloat16, device=DEV)
    k[:, at] = gap / d ** 0.5
    c.cache.write(k, _tokens("sink v", S, L, H, d), L, None, _i32(c.lens))


def _clear_values(c, blocks, zero_scale):
    """Zero values in these blocks: as the write leaves them, or with a scale of zero."""
    if zero_scale:
        c.cache.vs[:, :, blocks] = 0
    else:
        for j in blocks:
            c.cache.v[:, :, 64 * j:64 * j + 64].view(torch.uint8).zero_()
            c.cache.vs[:, :, j] = 2.0 ** -100


@pytest.mark.parametrize("rows", ROWS, ids=str)
@pytest.mark.parametrize("fmt", FORMATS)
def test_a_sink_whose_block_holds_no_values(fmt, rows):
    """The block of a row's far largest score has values of zero: the others' small weights are all of the output.
    Their largest weight times its scale is brought to 2^1 or more (2^8 where it lies within 2^-119 of the largest
    weight), so fp16's absolute half step of 2^-25 is 2^-26 of it."""
    N, G = rows
    for gap in (20.0, 78.0, 82.0, 85.0, 87.0, 90.0):
        for zero_scale in (True, False):
            for big in (0, 60, 100):  # other blocks' value scales up to 2^100
                c = DecodeCase(("sv", fmt, rows), fmt, 2, N, G, 1, 128, 16, 330, 0, [400] * (2 * N), [330, 270],
                               b_std=0.0, poison=False)
                _sink(c, 3, gap)
                c.cache.vs[:] = torch.exp2(torch.tensor([0.0, big, big - 8, big, big - 30, big - 3], device=DEV))
                _clear_values(c, [0], zero_scale)
                _check(c, c.run(), (gap, zero_scale, big), weight=12.0, floor=2.0 ** -26)


@pytest.mark.parametrize("rows", ROWS, ids=str)
@pytest.mark.parametrize("fmt", FORMATS)
def test_no_values_until_a_short_last_block(fmt, rows):
    """Zero values, then a last block of so few keys that half of its tile is past the end: large scores, and value
    scales 2^100 and more apart."""
    N, G = rows
    for lens in ([321, 286], [257, 342], [352, 353]):  # 5 or 6 tiles: a warp takes the last one and an earlier one
        for size, scale in ((3.0, 1.0), (1.0, 2.0 ** 60), (0.0, 2.0 ** 100)):
            for zero_scale in (True, False):
                c = DecodeCase(("lv", fmt, rows, lens), fmt, 2, N, G, 2, 64, 8, 384, 1, [0] * (2 * N), lens, b_std=0.0)
                c.q[:] = 1.0
                k = torch.full((2, 384, 2, 64), size * 12.0, dtype=torch.bfloat16, device=DEV)  # 96 * size a score
                c.cache.write(k, _tokens("lv v", 2, 384, 2, 64), 384, None, _i32(lens))
                last = [(n - 1) // 64 for n in lens]
                c.cache.vs[:] = scale
                for s, j in enumerate(last):
                    one = DecodeCase.__new__(DecodeCase)
                    one.cache = type("Part", (), dict(v=c.cache.v[s:s + 1], vs=c.cache.vs[s:s + 1]))
                    _clear_values(one, list(range(j)), zero_scale)
                # scores up to 288: 4 * 128 * 288 * 2^-24 = 36 * 2^-12
                _check(c, c.run(), (lens, size, scale, zero_scale), weight=36.0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_zero_values_as_written_before_large_ones(fmt):
    """All through the write: blocks of zeros (scale 2^-100), then 20 rows of about 2^30."""
    c = DecodeCase(("wr", fmt), fmt, 1, 2, 4, 1, 128, 16, 384, 0, [340, 340], [340], b_std=0.0)
    v = torch.zeros((1, 384, 1, 128), dtype=torch.bfloat16, device=DEV)
    v[:, 320:] = _tokens("wr v", 1, 64, 1, 128) * 2.0 ** 30
    c.cache.write(_tokens("wr k", 1, 384, 1, 128), v, 384, None, _i32([340]))
    _check(c, c.run(), fmt)


# ---------------------------------------------------------------------------
# one workspace for several shapes and operators
# ---------------------------------------------------------------------------

def _wide(seed, fmt="e4m3", S=40):
    """Many short sessions and a long last one: its items, past the 64th, are split over CTAs."""
    return DecodeCase(seed, fmt, S, 1, 8, 2, 64, 16, 4000, 1, [0] * S, [1 + i % 70 for i in range(S - 1)] + [4000])


def test_a_workspace_serves_a_growing_batch():
    wide = _wide("grow")
    want = wide.run()
    _check(wide, want, "wide")
    small = [DecodeCase(("grow", n), "int8", n, 2, 4, 1, 128, 32, 6000, 0, [0, 100] * n, [6000] * n)
             for n in (1, 2, 7)]
    ws = torch.zeros(max(c.workspace().numel() for c in small + [wide]), dtype=torch.uint8, device=DEV)
    for c in small:
        first = c.run()
        assert torch.equal(c.run(ws=ws), first)
        assert torch.equal(wide.run(ws=ws), want)
        assert torch.equal(c.run(ws=ws), first)


def test_a_workspace_that_other_operators_used():
    wide = _wide("others")
    want = wide.run()
    S, N, Hq, Hkv, d, r, L = 2, 8, 16, 2, 128, 16, 3000
    prob = lrkv.make_problem(S, N, Hq, Hkv, d, r)
    x = torch.randn((2, S, Hkv, L, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    kv = lrkv.kv_view_dense(x[0], x[1])
    u = torch.randn((S, N, L, r), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    b = torch.randn((N, r, Hkv * d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    T = 128
    q = torch.randn((N, T, Hq, d), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)
    one = torch.empty((S, N, Hq, d), dtype=torch.bfloat16, device=DEV)
    chunk = torch.empty_like(q)
    need = [lrkv.lrkv_decode_workspace_bytes(prob, L), lrkv.lrkv_prefill_workspace_bytes(prob, L - T, T)]
    ws = torch.zeros(max(need + [wide.workspace().numel()]), dtype=torch.uint8, device=DEV)
    lrkv.lrkv_attn_decode(prob, q[:S, 0].reshape(S, 1, Hq, d).repeat(1, N, 1, 1), kv, _i32([L, L]), L, u, b, None, one,
                          ws)
    assert torch.equal(wide.run(ws=ws), want)
    ws.zero_()
    lrkv.lrkv_attn_prefill_chunk(prob, q, kv, 0, L - T, T, u, b, None, chunk, ws)
    assert torch.equal(wide.run(ws=ws), want)
