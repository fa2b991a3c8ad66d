"""The 8-bit K/V cache on the GPU against its fp64 oracle.

Writing is compared code for code and scale for scale.  Reading back and decode
take tolerances that count roundings:

* read back: code * scale in fp32 (2^-24) and one bf16 rounding (2^-8 of the value);
* decode, fp32 output: each weight p enters the value product as fp16 (half a step,
  2^-11; the scaling before it 2^-22 or so) and the low-rank product as bf16 (2^-8).
  Scores are fp32 sums of at most 128 products, so a weight's exponent is off by
  at most 128 * 2^-24 * sum |q k| scale, under 2^-14 * max(1, sum |q k| scale / 8);
  numerator and denominator both carry it.  With A_v = sum p |v| and A_z = sum p |U| |B|:
  |err| <= 2^-11 A_v + 2^-8 A_z + 2^-12 (A_v + A_z) on data of unit size.
* A weight that is small beside its row's largest (p sv, with the block's value
  scale) meets fp16's absolute half step of 2^-25 below 2^-14.  The largest p sv is
  brought to 2^8 or more, so that is 2^-33 of it for every key, times the key's
  code: |err| <= ... + 2^-33 max_t(p sv) sum_t |code|.
* bf16 output: 2^-8 of the value more.
"""

import zlib

import numpy as np
import pytest
import torch

import lora_shared_kv_b200 as lrkv
import oracle
from oracle import kvq_oracle as kvq

pytestmark = pytest.mark.gpu

DEV = "cuda"
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def _seed(x):
    return zlib.crc32(str(x).encode()) % 100000


def _gen(x):
    g = torch.Generator(device="cpu")
    g.manual_seed(_seed(x))
    return g


def _numbers(codes):
    """Codes of a tensor as float64 numbers."""
    c = codes.cpu()
    if c.dtype == torch.int8:
        return c.double().numpy()
    return kvq.e4m3_from_bits(c.view(torch.uint8).numpy())


def _flags_ws():
    return torch.zeros(lrkv.KV_QUANT_WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)


class Cache:
    """An 8-bit cache of S sessions on the GPU, dense or paged, with its logical contents."""

    def __init__(self, fmt, S, Hkv, rows, d, paged=False, seed=0, spare=3, pad=0):
        g = _gen(("cache", fmt, S, Hkv, rows, d, paged, seed))
        nb = -(-rows // 64)
        self.fmt, self.S, self.Hkv, self.rows, self.d, self.paged = fmt, S, Hkv, rows, d, paged
        if paged:
            P = S * nb + spare
            self.table_cpu = torch.randperm(P, generator=g)[:S * nb].view(S, nb).to(torch.int32)
            self.table = self.table_cpu.to(DEV)
            cs, ss = (P, Hkv, 64, d + pad), (P, Hkv)
        else:
            cs, ss = (S, Hkv, rows, d + pad), (S, Hkv, nb)
        # anything may stand where nothing was written: random codes, NaN scales
        junk = torch.randint(0, 256, (2,) + cs, generator=g, dtype=torch.int32).to(torch.uint8).to(DEV)
        self.k, self.v = (junk[i].view(DTYPE[fmt])[..., :d] for i in range(2))
        self.ks, self.vs = (torch.full(ss, float("nan"), device=DEV) for _ in range(2))

    def view(self):
        if self.paged:
            return lrkv.kv_view_quant_paged(self.k, self.v, self.ks, self.vs, self.table)
        return lrkv.kv_view_quant_dense(self.k, self.v, self.ks, self.vs)

    def logical(self, which):
        """Codes' numbers [S, Hkv, rows, d] and scales [S, Hkv, blocks] in float64."""
        c, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        c, s = _numbers(c), s.double().cpu().numpy()
        if not self.paged:
            return c, s
        t = self.table_cpu.long().numpy()
        c = c[t].transpose(0, 2, 1, 3, 4).reshape(self.S, self.Hkv, -1, self.d)[:, :, :self.rows]
        return c, s[t].transpose(0, 2, 1)

    def problem(self, N=1, G=1, r=16, mode=0):
        return lrkv.make_problem(self.S, N, self.Hkv * G, self.Hkv, self.d, r, mode)

    def write(self, k, v, T, first=None, count=None, check="LRKV_OK"):
        """k, v [S, T, Hkv, d] (bf16 on the GPU)."""
        ws = _flags_ws()
        src = lrkv.kv_view_dense(k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3))
        lrkv.lrkv_quantize_kv(self.problem(), src, T, self.view(), self.rows, first, count, ws)
        st, flags = lrkv.lrkv_query_device_status(ws)
        assert st == check, (st, hex(flags))
        return flags


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _tokens(seed, S, T, H, d, spread=1.0):
    g = _gen(seed)
    size = torch.exp(spread * torch.randn((S, T, H, 1), generator=g))
    return (torch.randn((S, T, H, d), generator=g) * size).to(torch.bfloat16).to(DEV)


def _same(got, want):
    return np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


def _check_write(cache, before, k, v, first, count):
    """The cache holds what the oracle's write of the same tokens leaves, and nothing else moved."""
    for which, x in (("k", k), ("v", v)):
        codes, scales = (a.copy() for a in before[which])
        for s in range(cache.S):
            kvq.write(codes[s], scales[s], x[s, :count[s]].double().cpu().numpy(), first[s], cache.fmt)
        got_c, got_s = cache.logical(which)
        assert _same(got_s, scales), which
        assert _same(got_c, codes), which


WRITES = [  # S, Hkv, rows, d, T, first, count
    (1, 1, 64, 64, 1, [0], [1]),
    (1, 2, 200, 128, 200, [0], [200]),
    (3, 2, 300, 128, 100, [0, 63, 200], [100, 100, 100]),
    (4, 3, 257, 64, 130, [0, 1, 64, 127], [130, 0, 65, 130]),
    (2, 1, 129, 128, 1, [63, 128], [1, 1]),
    (5, 8, 70, 128, 2, [0, 62, 63, 64, 68], [2, 2, 2, 1, 2]),
]


@pytest.mark.parametrize("paged", [False, True], ids=["dense", "paged"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("shape", WRITES, ids=range(len(WRITES)))
def test_write_is_the_oracles_code_for_code(shape, fmt, paged):
    S, H, rows, d, T, first, count = shape
    cache = Cache(fmt, S, H, rows, d, paged)
    if any(f % 64 for f in first):  # the older rows of a block that is written into
        cache.write(_tokens(("old", shape), S, max(first), H, d), _tokens(("old v", shape), S, max(first), H, d),
                    max(first), None, _i32(first))
    before = {w: cache.logical(w) for w in "kv"}
    k, v = _tokens(("k", shape), S, T, H, d), _tokens(("v", shape), S, T, H, d)
    cache.write(k, v, T, _i32(first), _i32(count))
    _check_write(cache, before, k, v, first, count)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_token_by_token(fmt):
    """A cache that grows one token a call, with sizes that make the scales grow inside blocks."""
    S, H, d, n = 2, 2, 64, 70
    cache = Cache(fmt, S, H, 128, d, paged=True)
    state = {w: cache.logical(w) for w in "kv"}
    x = {w: _tokens((w, fmt, "grow"), S, n, H, d, spread=2.0) for w in "kv"}
    for t in range(n):
        cache.write(x["k"][:, t:t + 1], x["v"][:, t:t + 1], 1, _i32([t, t]), None)
        for w in "kv":
            for s in range(S):
                kvq.write(state[w][0][s], state[w][1][s], x[w][s, t:t + 1].double().cpu().numpy(), t, fmt)
    for w in "kv":
        got_c, got_s = cache.logical(w)
        assert _same(got_s, state[w][1]) and _same(got_c, state[w][0])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_every_bf16_magnitude_gets_its_scale(fmt):
    """One block per value: every bf16 magnitude as a block's largest element, next to ties and small elements."""
    bits = torch.arange(0, 0x7F80, 7, dtype=torch.int32)
    a = bits.to(torch.int16).view(torch.bfloat16)
    n = a.numel()
    x = torch.zeros((1, n * 64, 1, 64), dtype=torch.bfloat16)
    x[0, ::64, 0, 0] = a
    x[0, ::64, 0, 1] = -a
    x[0, 5::64, 0, 2:34] = (a.float()[:, None] * torch.arange(1, 33) / 64).to(torch.bfloat16)
    cache = Cache(fmt, 1, 1, n * 64, 64)
    before = {w: cache.logical(w) for w in "kv"}
    x = x.to(DEV)
    # the product a * k above passes fp32's range for the largest a: those elements are infinities
    assert torch.isinf(x).any()
    assert cache.write(x, x, n * 64, None, None, check="LRKV_ERR_DEVICE_FAULT") == 0x10
    _check_write(cache, before, x, x, [0], [n * 64])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_infinities_and_nans_are_flagged_and_leave_the_rest(fmt):
    S, H, d = 1, 2, 64
    k = _tokens("inf", S, 64, H, d)
    k[0, 3, 0, 5], k[0, 9, 0, 6], k[0, 20, 0, 7] = float("inf"), float("-inf"), float("nan")
    v = _tokens("fine", S, 64, H, d)
    cache = Cache(fmt, S, H, 64, d)
    before = {w: cache.logical(w) for w in "kv"}
    flags = cache.write(k, v, 64, None, None, check="LRKV_ERR_DEVICE_FAULT")
    assert flags == 0x10
    _check_write(cache, before, k, v, [0], [64])
    c, _ = cache.logical("k")
    top = kvq.TOP[fmt]
    assert c[0, 0, 3, 5] == top and c[0, 0, 9, 6] == -top
    assert np.isnan(c[0, 0, 20, 7]) if fmt == "e4m3" else c[0, 0, 20, 7] == 0


def test_strides_sources_and_paged_sources():
    """Head-major, token-major, padded and paged bf16 sources give the same cache."""
    S, H, d, T = 2, 3, 128, 150
    k, v = _tokens("s k", S, T, H, d), _tokens("s v", S, T, H, d)
    got = []
    for layout in range(4):
        cache = Cache("e4m3", S, H, 200, d, pad=16 if layout == 2 else 0)
        ws = _flags_ws()
        if layout == 0:
            src = lrkv.kv_view_dense(k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3))
        elif layout == 1:
            src = lrkv.kv_view_dense(k.permute(0, 2, 1, 3).contiguous(), v.permute(0, 2, 1, 3).contiguous())
        elif layout == 2:
            wide = torch.full((2, S, T, H, d + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
            wide[0, ..., :d], wide[1, ..., :d] = k, v
            src = lrkv.kv_view_dense(wide[0].permute(0, 2, 1, 3)[..., :d], wide[1].permute(0, 2, 1, 3)[..., :d])
        else:
            pages = torch.full((2, 2 * S * 3, H, 64, d), float("nan"), dtype=torch.bfloat16, device=DEV)
            table = torch.randperm(2 * S * 3, generator=_gen("pages"))[:S * 3].view(S, 3)
            for s in range(S):
                for j in range(3):
                    n = min(64, T - 64 * j)
                    for i, x in enumerate((k, v)):
                        pages[i, table[s, j], :, :n] = x[s, 64 * j:64 * j + n].permute(1, 0, 2)
            table = table.to(torch.int32).to(DEV)
            src = lrkv.kv_view_paged(pages[0], pages[1], table)
        lrkv.lrkv_quantize_kv(cache.problem(), src, T, cache.view(), 200, _i32([0, 0]), None, ws)
        assert lrkv.lrkv_query_device_status(ws)[0] == "LRKV_OK"
        got.append([a[:, :, :T] if a.ndim == 4 else a for w in "kv" for a in cache.logical(w)])
    for other in got[1:]:
        assert all(_same(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("paged", [False, True], ids=["dense", "paged"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("shape", WRITES[1:], ids=range(len(WRITES) - 1))
def test_read_back(shape, fmt, paged):
    S, H, rows, d, T, first, count = shape
    cache = Cache(fmt, S, H, rows, d, paged)
    cache.write(_tokens(("rk", shape), S, rows, H, d), _tokens(("rv", shape), S, rows, H, d), rows, None, None)
    out = torch.full((2, S, H, T + 3, d), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = _flags_ws()
    lrkv.lrkv_dequantize_kv(cache.problem(), cache.view(), rows, T, lrkv.kv_view_dense(out[0], out[1]), _i32(first),
                            _i32(count), ws)
    assert lrkv.lrkv_query_device_status(ws)[0] == "LRKV_OK"
    for i, w in enumerate("kv"):
        y = kvq.values(*cache.logical(w))
        got = out[i].double().cpu().numpy()
        for s in range(S):
            n = count[s]
            want = y[s, :, first[s]:first[s] + n]
            assert np.all(np.abs(got[s, :, :n] - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23))
            if fmt == "e4m3":
                assert np.array_equal(got[s, :, :n], want)  # 4 bits times a power of two
            assert np.all(got[s, :, n:] == 7.0)


def test_read_into_pages():
    S, H, d, T = 2, 2, 128, 130
    cache = Cache("e4m3", S, H, T, d)
    cache.write(_tokens("pk", S, T, H, d), _tokens("pv", S, T, H, d), T, None, None)
    pages = torch.full((2, 9, H, 64, d), 7.0, dtype=torch.bfloat16, device=DEV)
    table_cpu = torch.randperm(9, generator=_gen("into"))[:6].view(S, 3)
    table = table_cpu.to(torch.int32).to(DEV)
    ws = _flags_ws()
    lrkv.lrkv_dequantize_kv(cache.problem(), cache.view(), T, T, lrkv.kv_view_paged(pages[0], pages[1], table), None,
                            None, ws)
    assert lrkv.lrkv_query_device_status(ws)[0] == "LRKV_OK"
    for i, w in enumerate("kv"):
        y = kvq.values(*cache.logical(w))
        got = pages[i].double().cpu().numpy()[table_cpu.numpy()].transpose(0, 2, 1, 3, 4).reshape(S, H, 192, d)
        assert np.array_equal(got[:, :, :T], y) and np.all(got[:, :, T:] == 7.0)


def test_bad_ranges_and_pages_are_flagged_and_skipped():
    S, H, d = 4, 2, 64
    k, v = _tokens("bk", S, 20, H, d), _tokens("bv", S, 20, H, d)
    cache = Cache("int8", S, H, 100, d)
    before = {w: cache.logical(w) for w in "kv"}
    flags = cache.write(k, v, 20, _i32([-1, 81, 0, 5]), _i32([5, 20, 21, -3]), check="LRKV_ERR_DEVICE_FAULT")
    assert flags == 0x1
    for w in "kv":
        assert all(_same(a, b) for a, b in zip(cache.logical(w), before[w]))
    paged = Cache("e4m3", 2, H, 128, d, paged=True)
    paged.table[0, 1] = paged.k.shape[0]
    paged.table[1, 0] = -1
    x = _tokens("bp", 2, 128, H, d)
    flags = paged.write(x, x, 128, None, None, check="LRKV_ERR_DEVICE_FAULT")
    assert flags == 0x4
    out = torch.full((2, 2, H, 128, d), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = _flags_ws()
    lrkv.lrkv_dequantize_kv(paged.problem(), paged.view(), 128, 128, lrkv.kv_view_dense(out[0], out[1]), None, None,
                            ws)
    st, flags = lrkv.lrkv_query_device_status(ws)
    assert st == "LRKV_ERR_DEVICE_FAULT" and flags == 0x4
    assert (out[:, 0, :, 64:] == 7.0).all() and (out[:, 1, :, :64] == 7.0).all()
    assert (out[:, 0, :, :64] != 7.0).any() and (out[:, 1, :, 64:] != 7.0).any()


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

class DecodeCase:
    def __init__(self, seed, fmt, S, N, G, Hkv, d, r, L, mode, offs, lens, paged=False, spread=0.5, q_std=1.0,
                 b_std=0.05, poison=True):
        self.N, self.G, self.r, self.mode, self.L = N, G, r, mode, L
        self.cache = Cache(fmt, S, Hkv, L, d, paged, seed=_seed(seed))
        k, v = _tokens((seed, "k"), S, L, Hkv, d, 0.1), _tokens((seed, "v"), S, L, Hkv, d, spread)
        self.cache.write(k, v, L, None, _i32(lens))
        g = _gen((seed, "rest"))
        nu = N if mode == 0 else 1
        self.q = (torch.randn((S, N, Hkv * G, d), generator=g) * q_std).to(torch.bfloat16).to(DEV)
        u = torch.randn((S, nu, L, r), generator=g).to(torch.bfloat16)
        self.u_clean = u.double().numpy()
        self.offs = np.array(offs, dtype=np.int64).reshape(S, N)
        self.lens = lens
        if poison:  # rows that no agent uses
            for s in range(S):
                u[s, :, lens[s]:] = float("nan")
                for i in range(nu):
                    a = int(self.offs[s, i] if mode == 0 else self.offs[s].min())
                    u[s, i, :a] = float("nan")
        self.u = u.to(DEV)
        self.b = (torch.randn((N, r, Hkv * d), generator=g) * b_std).to(torch.bfloat16).to(DEV)
        self.problem = self.cache.problem(N, G, r, mode)

    def workspace(self):
        return torch.zeros(lrkv.lrkv_decode_quant_workspace_bytes(self.problem, self.L), dtype=torch.uint8, device=DEV)

    def run(self, dtype=torch.float32, ws=None, offsets=True, check=True, stream=None):
        ws = self.workspace() if ws is None else ws
        out = torch.full(self.q.shape, float("nan"), dtype=dtype, device=DEV)
        lrkv.lrkv_attn_decode_quant(self.problem, self.q, self.cache.view(), _i32(self.lens), self.L, self.u, self.b,
                                    _i32(self.offs.tolist()) if offsets else None, out, ws, stream=stream)
        if check:
            st, flags = lrkv.lrkv_query_device_status(ws)
            assert st == "LRKV_OK", (st, hex(flags))
        return out

    def reference(self):
        k, v = (np.nan_to_num(kvq.values(*self.cache.logical(w)), nan=0.0, posinf=0.0, neginf=0.0) for w in "kv")
        sv = np.nan_to_num(self.cache.logical("v")[1])
        return kvq.decode_with_bound(self.q.double().cpu().numpy(), k, v, self.u_clean, self.b.double().cpu().numpy(),
                                     self.offs, self.lens, self.mode, sv)

    def check(self, out, what="", weight=1.0):
        ref, a_v, a_z, floor = self.reference()
        got = out.double().cpu().numpy()
        assert np.all(np.isfinite(got)), what
        bound = 2.0 ** -11 * a_v + 2.0 ** -8 * a_z + weight * 2.0 ** -12 * (a_v + a_z) + 2.0 ** -33 * floor
        if out.dtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * np.abs(ref)
        worst = np.max(np.abs(got - ref) / np.maximum(bound, 1e-30))
        assert worst <= 1.0, (what, worst)


SHAPES = [  # S, N, G, Hkv, d, r, L, mode, offsets, lens
    (1, 1, 1, 1, 64, 8, 1, 0, [0], [1]),
    (2, 2, 2, 1, 64, 8, 256, 0, [128, 192, 0, 300], [256, 64]),
    (1, 1, 8, 2, 128, 16, 130, 0, [65], [130]),                          # 8 rows, one agent
    (3, 2, 2, 2, 128, 16, 700, 1, [0, 100, 5, 5, 0, 0], [700, 1, 64]),   # 4 rows, shared U
    (2, 3, 3, 1, 128, 32, 333, 0, [0, 40, 333, 7, 64, 65], [333, 200]),  # 9 rows
    (2, 8, 2, 2, 128, 16, 515, 0, list(range(0, 512, 32)), [515, 129]),  # 16 rows, eight agents
    (2, 3, 6, 2, 128, 16, 1000, 0, [0, 300, 999, 17, 64, 2000], [1000, 777]),  # 18 rows
    (3, 4, 5, 1, 64, 16, 450, 0, [0, 7, 449, 100, 1, 1, 1, 1, 64, 65, 200, 0], [450, 1, 449]),  # 20 rows
    (2, 3, 8, 1, 128, 8, 260, 1, [0, 130, 259, 3, 3, 0], [260, 0]),      # 24 rows, an empty session
    (1, 5, 5, 1, 128, 32, 300, 0, [0, 10, 100, 200, 299], [300]),        # 25 rows: two row blocks
    (2, 16, 2, 1, 64, 32, 190, 0, list(range(0, 192, 6)), [190, 63]),    # 32 rows, 16 agents
    (1, 5, 8, 1, 64, 32, 300, 0, [0, 10, 100, 200, 299], [300]),         # 40 rows: two row groups
    (1, 8, 8, 1, 128, 16, 200, 1, [0, 3, 64, 65, 128, 199, 200, 500], [200]),  # 64 rows
    (1, 3, 7, 2, 128, 8, 129, 0, [0, 128, 129], [129]),                  # 21 rows, rank 8
    (5, 1, 1, 3, 128, 16, 4097, 0, [0, 4000, 4096, 1, 64], [4097, 63, 0, 64, 65]),  # ragged
    (1, 8, 2, 1, 128, 32, 1500, 0, [0, 1, 2, 3, 64, 700, 1400, 1499], [1500]),   # large U tiles: groups share stages
    (1, 16, 1, 1, 128, 32, 1100, 0, list(range(0, 1040, 65)), [1100]),           # one U stage for every group
    (41, 1, 2, 1, 64, 8, 150, 0, [(7 * i) % 160 for i in range(41)], [(i * 37) % 151 for i in range(41)]),  # 41 sessions
]


@pytest.mark.parametrize("paged", [False, True], ids=["dense", "paged"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"S{s[0]}N{s[1]}G{s[2]}H{s[3]}d{s[4]}r{s[5]}L{s[6]}m{s[7]}"
                                               for s in SHAPES])
def test_decode_shapes(shape, fmt, paged):
    c = DecodeCase(shape, fmt, *shape, paged=paged)
    out = c.run()
    for s, n in enumerate(c.lens):
        if n == 0:
            assert (out[s] == 0).all()
    c.check(out, str(shape))
    assert torch.equal(c.run(torch.bfloat16), out.to(torch.bfloat16))


def test_long_item_over_many_ctas():
    # one item of 300 tiles: every CTA holds a stretch of it, and the last merges up to 148 records
    c = DecodeCase("long", "e4m3", 1, 3, 6, 1, 128, 16, 19200, 0, [0, 9000, 19000], [19200])
    c.check(c.run(), "long")
    # a session far longer than the others
    c = DecodeCase("skew", "int8", 6, 2, 2, 1, 64, 16, 9000, 0, [0] * 12, [1, 64, 9000, 0, 65, 300], paged=True)
    c.check(c.run(), "skew")


def test_paged_is_dense_bit_for_bit_and_runs_repeat():
    shape = (3, 4, 2, 2, 128, 16, 576, 0, [0, 100, 576, 200, 64, 65, 300, 1, 500, 0, 0, 0], [576, 500, 33])
    a = DecodeCase("pd", "e4m3", *shape)
    b = DecodeCase("pd", "e4m3", *shape, paged=True)
    ws = a.workspace()
    first = a.run(ws=ws)
    assert torch.equal(first, a.run(ws=ws))
    assert torch.equal(first, b.run())


def test_sessions_that_share_pages():
    """Two sessions whose page tables begin with the same pages, and a page that a table names twice."""
    c = DecodeCase("share", "e4m3", 2, 2, 2, 2, 128, 16, 320, 0, [0, 64, 0, 64], [320, 320], paged=True)
    c.cache.table[1, :3] = c.cache.table[0, :3]
    c.cache.table[1, 4] = c.cache.table[1, 3]
    c.cache.table_cpu = c.cache.table.cpu()
    c.check(c.run(), "shared pages")


def test_two_streams_with_their_own_workspaces():
    a = DecodeCase("stream a", "e4m3", 2, 3, 2, 2, 128, 16, 2000, 0, [0, 900, 1999, 7, 64, 65], [2000, 1500])
    b = DecodeCase("stream b", "int8", 3, 2, 4, 1, 64, 32, 1700, 1, [0, 5, 0, 0, 1, 2], [1700, 3, 900], paged=True)
    want = [a.run(), b.run()]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [a.workspace(), b.workspace()]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        for case, st, ws in zip((a, b), streams, spaces):
            with torch.cuda.stream(st):
                outs.append(case.run(ws=ws, check=False))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 2])
    assert all(lrkv.lrkv_query_device_status(ws)[0] == "LRKV_OK" for ws in spaces)


def test_views_too_small_are_refused():
    c = DecodeCase("small", "int8", 2, 2, 2, 2, 64, 16, 100, 0, [0, 0, 0, 0], [100, 100])
    c.L = 101
    with pytest.raises(ValueError, match="8-bit view holds"):
        lrkv.lrkv_attn_decode_quant(c.problem, c.q, c.cache.view(), _i32(c.lens), 101, c.u, c.b, None,
                                    torch.empty_like(c.q), c.workspace())
    k = _tokens("small", 2, 5, 2, 64)
    with pytest.raises(ValueError, match="bf16 view holds"):
        c.cache.write(k, k, 6, None, None)
    wide = lrkv.make_problem(2, 1, 3, 3, 64, 16)
    src = lrkv.kv_view_dense(k.permute(0, 2, 1, 3), k.permute(0, 2, 1, 3))
    with pytest.raises(ValueError, match="view holds"):
        lrkv.lrkv_dequantize_kv(wide, c.cache.view(), 100, 5, src, None, None, _flags_ws())
    with pytest.raises(ValueError, match="int32"):
        lrkv.lrkv_quantize_kv(c.problem, src, 5, c.cache.view(), 100, _i32([0, 0]).long(), None, _flags_ws())


def test_no_tokens_at_all_and_bounds_below_the_cache():
    c = DecodeCase("none", "e4m3", 2, 2, 2, 2, 64, 16, 300, 0, [0, 0, 0, 0], [300, 200])
    c.lens, c.L = [0, 0], 0
    assert (c.run() == 0).all()
    c.lens, c.L = [70, 0], 100  # the bound is the call's, not the cache's
    c.check(c.run(), "bound below the cache")


def test_every_code_enters_as_the_number_it_is():
    for fmt in ("int8", "e4m3"):  # int8's -128 is not written, but read
        c = DecodeCase("codes", fmt, 1, 1, 4, 1, 128, 16, 192, 0, [192], [192])
        codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
        if fmt == "e4m3":
            codes = codes[(codes & 0x7F) != 0x7F]  # without the NaNs
        n = 192 * 128
        for i, t in enumerate((c.cache.k, c.cache.v)):
            t.view(torch.uint8).copy_(codes.repeat(n // codes.numel() + 1)[i:i + n].view(1, 1, 192, 128).to(DEV))
        c.cache.ks[:] = 2.0 ** -7 if fmt == "int8" else 2.0 ** -9
        c.cache.vs[:] = 2.0 ** -5
        c.check(c.run(), fmt)


def test_null_offsets_are_zero():
    c = DecodeCase("null", "e4m3", 2, 2, 2, 2, 128, 16, 333, 0, [0, 0, 0, 0], [333, 200])
    assert torch.equal(c.run(), c.run(offsets=False))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_value_scales_far_apart(fmt):
    """Blocks whose value scales differ by up to 2^70: each row's own reference keeps its small weights."""
    c = DecodeCase("apart", fmt, 2, 2, 8, 1, 128, 16, 640, 0, [0, 640, 0, 0], [640, 600], b_std=0.0)
    for e in ([-60, 10, -20, 0, 8, -1, 3, -60, 2, -3], [0, -50, -50, 0, -45, -60, -60, -60, -60, -60]):
        c.cache.vs.copy_(torch.exp2(torch.tensor(e, dtype=torch.float32, device=DEV)).expand(2, 1, 10))
        c.check(c.run(), f"{e}")
    # blocks of scale zero hold zeros
    c.cache.vs[:, :, 3:7] = 0
    c.cache.vs[1] = 0
    c.check(c.run(), "zero value scales")
    c.cache.ks[:, :, 2:5] = 0
    c.check(c.run(), "zero key scales")


def test_a_sink_and_a_long_flat_tail():
    """One key 2^20 above the rest of a long context whose small weights add up: none may be lost."""
    L = 16384
    c = DecodeCase("sink", "e4m3", 1, 1, 4, 1, 64, 8, L, 0, [L], [L], spread=0.0, b_std=0.0)
    c.q[:] = 1.0
    x = torch.zeros((1, L, 1, 64), dtype=torch.bfloat16, device=DEV)
    x[:, 7] = 20 * 0.6931 * 8 / 64          # score 20 ln 2 against 0
    v = torch.ones((1, L, 1, 64), dtype=torch.bfloat16, device=DEV)
    v[:, 7] = 0
    c.cache.write(x, v, L, None, None)
    # p of the tail: 16383 / (2^20 + 16383) = 0.0154, all of the output
    c.check(c.run(), "sink")


def test_large_scores_and_queries():
    # sum |q k| scale is about 128 * 24 * 0.8 / 11.3 = 217 here: an exponent is off by at most 128 * 217 * 2^-24 =
    # 1.7e-3, twice that where the tensor cores truncate, and again for the denominator: 6.6e-3 = 27 * 2^-12
    c = DecodeCase("large", "int8", 1, 2, 4, 1, 128, 16, 300, 0, [0, 150], [300], q_std=30.0)
    c.check(c.run(), "large", weight=40.0)
    for f in (2.0 ** 100, 2.0 ** -100):  # the queries' own size cancels against the softmax scale
        d = DecodeCase("scaled q", "e4m3", 1, 2, 4, 1, 128, 16, 300, 0, [0, 150], [300])
        want = d.run()
        d.q = (d.q.double() * f).to(torch.bfloat16)
        d.problem.softmax_scale = float(1 / np.sqrt(128.0) / f)
        assert torch.equal(d.run(), want)


def test_strided_caches():
    c = DecodeCase("strided", "e4m3", 2, 2, 3, 2, 64, 16, 200, 0, [0, 50, 0, 0], [200, 131])
    want = c.run()
    wide = torch.full((2, 2, 230, 2, 96), 0x7F, dtype=torch.uint8, device=DEV)  # NaN between the rows
    for i, t in enumerate((c.cache.k, c.cache.v)):
        wide[i, :, :200, :, 16:80] = t.view(torch.uint8).permute(0, 2, 1, 3)
    c.cache.k, c.cache.v = (wide[i].view(torch.float8_e4m3fn).permute(0, 2, 1, 3)[:, :, :200, 16:80] for i in range(2))
    sc = torch.full((2, 2, 2, 9), float("nan"), device=DEV)
    sc[0, :, :, :4], sc[1, :, :, :4] = c.cache.ks, c.cache.vs
    c.cache.ks, c.cache.vs = sc[0, :, :, :4], sc[1, :, :, :4]
    u = torch.full((2, 2, 250, 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    u[:, :, :200, :16] = c.u
    c.u = u[..., :16]
    assert torch.equal(c.run(), want)


def test_flags_instead_of_faults():
    c = DecodeCase("flags", "e4m3", 2, 2, 2, 2, 128, 16, 256, 0, [0, 5, 3, 3], [256, 256], paged=True)
    good = c.run()
    c.lens, c.offs = [256, 999], np.array([[0, -5], [3, 3]])
    ws = c.workspace()
    c.run(ws=ws, check=False)
    st, flags = lrkv.lrkv_query_device_status(ws)
    assert st == "LRKV_ERR_DEVICE_FAULT" and flags == 0x3
    assert lrkv.lrkv_query_device_status(ws) == ("LRKV_OK", 0)
    c.lens, c.offs = [256, 256], np.array([[0, 5], [3, 3]])
    keep = c.cache.table.clone()
    c.cache.table[1, 2] = c.cache.k.shape[0]
    got = c.run(ws=ws, check=False)
    st, flags = lrkv.lrkv_query_device_status(ws)
    assert st == "LRKV_ERR_DEVICE_FAULT" and flags == 0x4
    assert torch.equal(got[0], good[0]) and torch.isfinite(got).all()
    c.cache.table.copy_(keep)
    assert torch.equal(c.run(ws=ws), good)


def test_a_wait_that_runs_out_is_reported():
    c = DecodeCase("stall", "int8", 2, 3, 6, 2, 128, 16, 640, 0, [0, 300, 639, 17, 64, 2000], [640, 333])
    ws = c.workspace()
    want = c.run(ws=ws)
    lrkv.lrkv_debug_stall_next_launch(4)
    c.run(ws=ws, check=False)
    assert lrkv.lrkv_query_device_status(ws)[0] == "LRKV_ERR_TIMEOUT"
    lrkv.lrkv_workspace_reset(ws)
    assert torch.equal(c.run(ws=ws), want)


def test_a_captured_serving_step_replays_on_new_data():
    """Write one token per session and decode, captured once; two graphs share one workspace on one stream."""
    S, N, G, H, d, r, L = 3, 2, 3, 2, 128, 16, 300
    lens = [100, 191, 7]
    a = DecodeCase("graph", "e4m3", S, N, G, H, d, r, L, 0, [0, 50, 90, 0, 0, 3], lens)
    pos, sl, offs = _i32(lens), _i32([n + 1 for n in lens]), _i32(a.offs.tolist())
    k, v = _tokens("gk", S, 1, H, d), _tokens("gv", S, 1, H, d)
    a.u = torch.from_numpy(a.u_clean).to(torch.bfloat16).to(DEV)
    ws, fws = a.workspace(), _flags_ws()
    view, src = a.cache.view(), lrkv.kv_view_dense(k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3))
    out = torch.zeros(a.q.shape, dtype=torch.float32, device=DEV)

    def step():
        lrkv.lrkv_quantize_kv(a.problem, src, 1, view, L, pos, None, fws)
        lrkv.lrkv_attn_decode_quant(a.problem, a.q, view, sl, L, a.u, a.b, offs, out, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        before = [t.clone() for t in (a.cache.k.view(torch.uint8), a.cache.v.view(torch.uint8), a.cache.ks, a.cache.vs)]
        step()
        for t, b in zip((a.cache.k.view(torch.uint8), a.cache.v.view(torch.uint8), a.cache.ks, a.cache.vs), before):
            t.copy_(b)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g, stream=side):
            step()
            pos.add_(1)
            sl.add_(1)
    for i in range(4):
        k.copy_(_tokens(("gk", i), S, 1, H, d))
        v.copy_(_tokens(("gv", i), S, 1, H, d))
        a.q.copy_(torch.randn(a.q.shape, generator=_gen(("gq", i))).to(torch.bfloat16))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[i % 2].replay()
        torch.cuda.synchronize()
        a.lens = [n + 1 + i for n in lens]
        a.check(out, f"replay {i}")
    assert lrkv.lrkv_query_device_status(ws)[0] == "LRKV_OK" and lrkv.lrkv_query_device_status(fws)[0] == "LRKV_OK"


def test_a_role_switch_over_an_8_bit_cache():
    """Write a chunk, read the context back, and run the prefill chunk over it."""
    N, G, H, d, r, L0, T = 2, 2, 2, 128, 16, 150, 70
    L = L0 + T
    cache = Cache("e4m3", 1, H, L, d, paged=True)
    cache.write(_tokens("ck", 1, L0, H, d, 0.1), _tokens("cv", 1, L0, H, d, 0.1), L0, None, None)
    cache.write(_tokens("nk", 1, T, H, d, 0.1), _tokens("nv", 1, T, H, d, 0.1), T, _i32([L0]), None)
    g = _gen("switch")
    q = torch.randn((N, T, H * G, d), generator=g).to(torch.bfloat16).to(DEV)
    u = torch.randn((1, N, L, r), generator=g).to(torch.bfloat16).to(DEV)
    b = (torch.randn((N, r, H * d), generator=g) * 0.05).to(torch.bfloat16).to(DEV)
    offs = _i32([0, 170])
    prob = lrkv.make_problem(1, N, H * G, H, d, r, 0)
    staged = torch.empty((2, 1, H, L, d), dtype=torch.bfloat16, device=DEV)
    back = lrkv.kv_view_dense(staged[0], staged[1])
    ws = torch.zeros(max(256, lrkv.lrkv_prefill_workspace_bytes(prob, L0, T)), dtype=torch.uint8, device=DEV)
    out = torch.empty((N, T, H * G, d), dtype=torch.bfloat16, device=DEV)
    lrkv.lrkv_dequantize_kv(prob, cache.view(), L, L, back, None, None, ws)
    lrkv.lrkv_attn_prefill_chunk(prob, q, back, 0, L0, T, u, b, offs, out, ws)
    assert lrkv.lrkv_query_device_status(ws)[0] == "LRKV_OK"
    k, v = (kvq.values(*cache.logical(w))[0] for w in "kv")
    want = oracle.prefill_chunk(q.cpu(), k, v, u[0].cpu(), b.cpu(), offs.cpu(), L0, 0)
    got = out.double().cpu().numpy()
    # the prefill chunk's own parity bar
    assert np.abs(got - want).max() <= 1e-2 and np.linalg.norm(got - want) / np.linalg.norm(want) <= 5e-3
