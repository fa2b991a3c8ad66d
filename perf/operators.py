"""Cases of the operators on a K/V cache held in 8 bits: writing it, reading it
back, and decode attention over it with per-agent low-rank values.

The cache holds one code of 8 bits per element (e4m3 or int8) and one fp32 scale
per block of 64 tokens and KV head, for K and for V.  An element stands for
code * scale.

``run`` computes a case in its plain form (elementary torch operations in 32 bits,
in 64 where a value next to a rounding border needs it) or, where ``own`` is true,
through lora_shared_kv_b200.  ``exact`` computes the same in 64 bits from the
definition, written separately.

Kinds of case:
  write   T new tokens per session are quantised into the cache
  read    rows of the cache are turned back into bf16
  decode  one query token per (session, agent) over the cache
  step    a serving step: one token per session is written, then decode
  chunk   a role switch: a chunk is written, the context is read back, and the
          chunk's rows attend to it (the causal prefill chunk)
"""

import math
import random

import torch

own = False

BLOCK = 64       # tokens of a block of the cache: one scale each for K and V and KV head
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100

DEV = "cuda"


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def _case(name, kind, fmt, S, Hkv, d, L, paged=False, T=1, start="end", N=1, G=1, r=16, shared_u=False,
          lens="full", offsets="late", src="tokens"):
    """L: rows of the cache per session.  lens: "full" (every session holds L rows) or "ragged" (1 .. L, one of
    them empty).  start: "end" (the new tokens are each session's last ones) or "zero".  offsets: "late" (in the
    second half of the context), "zero" (every token adapted).  src: layout of the new tokens, token-major as a
    projection gives them or head-major as a bf16 cache holds them."""
    c = dict(kind=kind, fmt=fmt, S=S, Hkv=Hkv, d=d, L=L, paged=paged, T=T, start=start, N=N, G=G, r=r,
             shared_u=shared_u, lens=lens, offsets=offsets, src=src)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # Long context, eight agents, 64-token pages in random order: the largest decode (0.55 GB of cache).
        _case("decode paged 64k 8 agents", "decode", "e4m3", 4, 8, 128, 65536, paged=True, N=8, G=2, r=16),
        # A coding team: three roles of a 12/2-head model, 32 sessions of 8k tokens (18 query rows per KV head).
        _case("decode 32x8k 3 roles", "decode", "int8", 32, 2, 128, 8192, N=3, G=6, r=16),
        # Short contexts, two specialists that share one U (4 query rows per KV head): launch costs matter.
        _case("decode 16x1k shared u", "decode", "e4m3", 16, 8, 128, 1024, N=2, G=2, r=16, shared_u=True,
              offsets="zero"),
        # Sessions of unequal lengths in pages, one of them empty, head_dim 64, rank 32, 20 rows per KV head.
        _case("decode ragged d64 r32", "decode", "int8", 24, 5, 64, 9001, paged=True, N=5, G=4, r=32, lens="ragged"),
        # The smallest call: one session, two agents, 256 tokens: latency.
        _case("decode tiny", "decode", "e4m3", 1, 1, 64, 256, N=2, G=2, r=8),
        # A 512-token chunk of one session joins a 16k context in the middle of a block.
        _case("write chunk 512", "write", "e4m3", 1, 8, 128, 16901, T=512),
        # A bf16 cache of four sessions is converted whole.
        _case("write bulk 4x16k", "write", "int8", 4, 8, 128, 16384, T=16384, start="zero", src="heads"),
        # Decode step's write: one token for each of 32 sessions, into pages.
        _case("write token x32", "write", "e4m3", 32, 8, 128, 2111, paged=True, T=1, lens="ragged"),
        # The context of a role switch is read back for the prefill chunk.
        _case("read 16k", "read", "e4m3", 1, 8, 128, 16384, T=16384, start="zero"),
        # Ragged tails of several sessions are read out of pages, head_dim 64.
        _case("read ragged tails d64", "read", "int8", 7, 3, 64, 1500, paged=True, T=300, lens="ragged"),
        # A whole serving step of the three-role team: write one token per session, then decode.
        _case("step 32x8k 3 roles", "step", "e4m3", 32, 2, 128, 8192, N=3, G=6, r=16),
        # A role switch: 512 rows of four agents on a 16k context held in 8 bits.
        _case("chunk 512 on 16k", "chunk", "e4m3", 1, 8, 128, 16896, T=512, N=4, G=2, r=32, offsets="zero"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))

    kind = rng.choice(["decode", "decode", "decode", "write", "write", "read", "step", "chunk"])
    fmt = rng.choice(["e4m3", "int8"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.randint(1, 8)
    paged = rng.random() < 0.5
    r = rng.choice([8, 16, 32])
    lens = rng.choice(["full", "ragged"])
    src = rng.choice(["tokens", "heads"])
    offsets = rng.choice(["late", "late", "zero"])
    shared_u = rng.random() < 0.3
    budget = 200e6  # bytes of codes a drawn cache holds at most
    if kind in ("decode", "step"):
        S = log_int(1, 48)
        L = log_int(1, int(min(65536, budget / (2 * S * Hkv * d))))
        return _case(None, kind, fmt, S, Hkv, d, L, paged, 1, "end", rng.randint(1, 8), rng.randint(1, 8), r,
                     shared_u, lens, offsets, src)
    if kind == "chunk":
        T = log_int(1, 512)
        L = T + log_int(1, 8192)
        return _case(None, kind, fmt, 1, Hkv, d, L, paged, T, "end", rng.randint(1, 4), rng.randint(1, 4), r,
                     shared_u, "full", offsets, src)
    S = log_int(1, 32)
    L = log_int(1, int(min(32768, budget / (2 * S * Hkv * d))))
    T = log_int(1, L)
    return _case(None, kind, fmt, S, Hkv, d, L, paged, T, rng.choice(["end", "zero"]), 1, 1, r, False, lens, "late",
                 src)


def _plan(c):
    """Host lists that a case fixes whatever the seed: lengths, rows written or read, offsets."""
    rng = random.Random("%(kind)s %(S)d %(L)d %(T)d %(N)d %(lens)s" % c)
    S, L, T = c["S"], c["L"], c["T"]
    if c["lens"] == "full":
        lens = [L] * S
    else:
        lens = [rng.randint(1, L) for _ in range(S)]
        lens[rng.randrange(S)] = L
        if c["kind"] == "decode" and S > 2:
            lens[rng.randrange(S)] = 0
    count = [min(T, n) for n in lens]
    first = [n - m for n, m in zip(lens, count)] if c["start"] == "end" else [0] * S
    offs = [[0 if c["offsets"] == "zero" else rng.randint(n // 2, n) for _ in range(c["N"])] for n in lens]
    return lens, first, count, offs


# ---------------------------------------------------------------------------
# the state of a user's program
# ---------------------------------------------------------------------------

def _pow2_ceil(x):
    """The smallest power of two >= x, for normal x > 0 (fp64, exact: made from the exponent's bits)."""
    m, e = torch.frexp(x.double())
    return ((torch.where(m == 0.5, e - 1, e).long() + 1023) << 52).view(torch.float64)


def _scale_for(amax, fmt):
    """The scale of a block whose largest finite magnitude is amax, in fp64: e4m3 takes the smallest power of two
    at which amax is at most 448 steps, int8 the smallest bf16 number at which it is at most 127."""
    a = amax.double()
    if fmt == "e4m3":
        s = _pow2_ceil(a.clamp_min(1e-300) / E4M3_MAX)
    else:
        t = (a / 127).float()
        s = ((t.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32).double()
        s = torch.where(s * 127 < a, (s.float().view(torch.int32) + 0x10000).view(torch.float32).double(), s)
        low = (s.float().view(torch.int32) - 0x10000).view(torch.float32).double()
        s = torch.where((low * 127 >= a) & (low > 0), low, s)
    return s.clamp_min(SCALE_MIN)


def _encode(y, fmt):
    """Codes of y (already divided by the scale): nearest, ties to even, saturating."""
    if fmt == "e4m3":
        return y.clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn)
    return y.round().clamp(-127, 127).to(torch.int8)


def _fresh_cache(c, x, gen):
    """Codes and scales of a filled cache: x is [S, Hkv, L, d] in bf16.  Rows past the end of a block stay 0."""
    S, H, L, d = x.shape
    nb = -(-L // BLOCK)
    f = torch.zeros((S, H, nb * BLOCK, d), dtype=torch.float32, device=DEV)
    f[:, :, :L] = x.float()
    f = f.view(S, H, nb, BLOCK, d)
    s = _scale_for(f.abs().amax(dim=(3, 4)), c["fmt"]).float()
    codes = _encode(f / s[..., None, None], c["fmt"])
    if not c["paged"]:
        return codes.view(S, H, nb * BLOCK, d)[:, :, :L].contiguous(), s.contiguous()
    # pages [S * nb, Hkv, 64, d] in the order of c's page table, scales [S * nb, Hkv]
    return codes.permute(0, 2, 1, 3, 4).reshape(S * nb, H, BLOCK, d), s.permute(0, 2, 1).reshape(S * nb, H)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7 + 3)
    S, H, d, L, T, N = c["S"], c["Hkv"], c["d"], c["L"], c["T"], c["N"]
    lens, first, count, offs = _plan(c)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)

    # keys with channels of unequal size, values whose size drifts along the context
    chan = torch.exp(0.5 * torch.randn((H, 1, d), generator=gen, device=DEV))
    drift = torch.exp(0.4 * torch.randn((S, H, -(-L // BLOCK), 1), generator=gen, device=DEV))
    drift = drift.expand(-1, -1, -1, BLOCK).reshape(S, H, -1)[:, :, :L, None]
    st = {"case": c, "max_len": max(1, max(lens))}
    nb = -(-L // BLOCK)
    if c["paged"]:
        perm = torch.randperm(S * nb, generator=gen, device=DEV)
        st["table"] = perm.view(S, nb).to(torch.int32)
    for name, mul in (("k", chan), ("v", drift)):
        codes, scale = _fresh_cache(c, (torch.randn((S, H, L, d), generator=gen, device=DEV) * mul).bfloat16(), gen)
        if c["paged"]:
            at = torch.empty_like(perm)
            at[perm] = torch.arange(S * nb, device=DEV)  # logical page held by each physical one
            codes, scale = codes.view(torch.uint8)[at].view(codes.dtype), scale[at].contiguous()
        st[name + "8"], st[name + "_scale"] = codes, scale
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["first"] = torch.tensor(first, dtype=torch.int32, device=DEV)
    st["count"] = torch.tensor(count, dtype=torch.int32, device=DEV)
    if c["kind"] in ("write", "step", "chunk"):  # the new tokens, some larger than what their block holds
        big = torch.exp(0.7 * torch.randn((S, T, H, 1), generator=gen, device=DEV))
        for name in ("k", "v"):
            x = (torch.randn((S, T, H, d), generator=gen, device=DEV) * big).bfloat16()
            if c["src"] == "heads":  # [S, T, Hkv, d] over head-major memory
                x = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
            st[name + "_new"] = x
    if c["kind"] in ("decode", "step", "chunk"):
        rows = (N, T) if c["kind"] == "chunk" else (S, N)
        st["q"] = normal(*rows, H * c["G"], d)
        st["u"] = normal(S, 1 if c["shared_u"] else N, L, c["r"])
        st["b"] = (0.05 * torch.randn((N, c["r"], H * d), generator=gen, device=DEV)).bfloat16()
        st["offsets"] = torch.tensor(offs, dtype=torch.int32, device=DEV).reshape(S, N)
        st["out"] = torch.empty((*rows, H * c["G"], d), dtype=torch.bfloat16, device=DEV)
    if c["kind"] in ("read", "chunk"):
        rows = L if c["kind"] == "chunk" else T
        st["k_out"] = torch.zeros((S, H, rows, d), dtype=torch.bfloat16, device=DEV)
        st["v_out"] = torch.zeros((S, H, rows, d), dtype=torch.bfloat16, device=DEV)
    return st


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _rows_at(st, s, t):
    """Index pair of the row of token t of session s in a cache's [*, row, Hkv, d] view."""
    if not st["case"]["paged"]:
        return s, t
    return st["table"].long()[s, t // BLOCK], t % BLOCK


def _write(st, name, x):
    """Write the new tokens x [S, T, Hkv, d] of one of K, V into its cache, in place."""
    c = st["case"]
    codes, scale, fmt = st[name + "8"], st[name + "_scale"], c["fmt"]
    S, T = x.shape[:2]
    first, count = st["first"].long()[:, None], st["count"].long()[:, None]
    nb = (T + 2 * BLOCK - 2) // BLOCK  # blocks that a session's rows can touch
    blk = first // BLOCK + torch.arange(nb, device=DEV)                             # [S, nb]
    t = (blk[:, :, None] * BLOCK + torch.arange(BLOCK, device=DEV)).view(S, -1)     # [S, nb * 64]
    s = torch.arange(S, device=DEV)[:, None].expand(t.shape)
    is_new = (t >= first) & (t < first + count)
    is_old = t < first
    touched = is_new.view(S, nb, BLOCK).any(2)
    top = st["table"].shape[1] * BLOCK if c["paged"] else codes.shape[2]
    a, b = _rows_at(st, s, t.clamp(0, top - 1))
    held = codes.view(torch.uint8).permute(0, 2, 1, 3)[a, b].view(codes.dtype).float()
    new = x[s, (t - first).clamp(0, T - 1)].float()
    H, d = new.shape[2:]
    fine = torch.where(torch.isfinite(new) & is_new[..., None, None], new.abs(), 0.0)
    need = _scale_for(fine.view(S, nb, BLOCK, H, d).amax(dim=(2, 4)), fmt).float()   # [S, nb, Hkv]
    blk_in = blk.clamp(0, -(-top // BLOCK) - 1)
    sa = (st["table"].long()[s[:, :nb], blk_in],) if c["paged"] else (s[:, :nb], blk_in)
    before = scale[sa] if c["paged"] else scale.permute(0, 2, 1)[sa]
    kept = is_old.view(S, nb, BLOCK).any(2)[..., None]
    after = torch.where(kept, torch.maximum(before, need), need)
    wide = lambda v: v[:, :, None].expand(S, nb, BLOCK, H).reshape(S, nb * BLOCK, H, 1).double()  # noqa: E731
    y = torch.where(is_new[..., None, None], new.double(), held.double() * wide(before)) / wide(after)
    fresh = _encode(y, fmt)
    put = (is_new | is_old) & touched[:, :, None].expand(S, nb, BLOCK).reshape(S, -1)
    codes.view(torch.uint8).permute(0, 2, 1, 3)[a[put], b[put]] = fresh.view(torch.uint8)[put]
    at = tuple(i[touched] for i in sa)
    (scale if c["paged"] else scale.permute(0, 2, 1))[at] = after[touched]


def _values(st, name, s, t):
    """What rows t [S, R] of K or V stand for: [S, R, Hkv, d] in fp32."""
    codes, scale = st[name + "8"], st[name + "_scale"]
    a, b = _rows_at(st, s, t)
    y = codes.view(torch.uint8).permute(0, 2, 1, 3)[a, b].view(codes.dtype).float()
    z = scale[a] if st["case"]["paged"] else scale.permute(0, 2, 1)[s, t // BLOCK]
    return y * z[..., None]


def _read(st, first, count, rows):
    """Rows [first, first + count) of every session as bf16 into the first rows of k_out and v_out."""
    S = st["lens"].numel()
    i = torch.arange(rows, device=DEV)[None]
    top = (st["table"].shape[1] * BLOCK if st["case"]["paged"] else st["k8"].shape[2]) - 1
    s = torch.arange(S, device=DEV)[:, None]
    live = (i < count[:, None])[:, None, :, None]
    for name in ("k", "v"):
        y = _values(st, name, s, (first.long()[:, None] + i).clamp(0, top)).bfloat16().permute(0, 2, 1, 3)
        st[name + "_out"][:, :, :rows] = torch.where(live, y, st[name + "_out"][:, :, :rows])
    return st["k_out"], st["v_out"]


def _attend(c, q, k, v, u, b, keep, use):
    """q [S, N, R, Hq, d] over k, v [S, Hkv, L, d], u [S, N, L, r], b [N, r, Hkv d].  keep [S, R, L]: the keys that
    row R sees; use [S, N, L]: the keys whose low-rank value counts.  A row that sees nothing gives 0."""
    S, N, R, Hq, d = q.shape
    H, G = c["Hkv"], c["G"]
    qg = q.float().view(S, N, R, H, G, d).permute(0, 3, 1, 4, 2, 5).reshape(S, H, N * G * R, d)
    sc = torch.matmul(qg, k.transpose(2, 3)) / math.sqrt(d)
    sc = sc.view(S, H, N, G, R, -1).masked_fill(~keep[:, None, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(torch.isfinite(m), m, 0.0))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    o = torch.matmul(p.view(S, H, N * G * R, -1), v).view(S, H, N, G, R, d)
    z = torch.matmul((p * use[:, None, :, None, None]).reshape(S, H, N, G * R, -1), u.float()[:, None])
    bh = b.float().view(N, -1, H, d).permute(2, 0, 1, 3)                              # [Hkv, N, r, d]
    o = o + torch.matmul(z, bh[None]).view(S, H, N, G, R, d)
    return o.permute(0, 2, 4, 1, 3, 5).reshape(S, N, R, Hq, d)


def _decode(st):
    c = st["case"]
    S, N, L = c["S"], c["N"], st["max_len"]
    pos = torch.arange(L, device=DEV)
    s = torch.arange(S, device=DEV)[:, None]
    live = pos[None] < st["lens"][:, None]                                            # [S, L]
    k = _values(st, "k", s, pos[None].expand(S, L)).permute(0, 2, 1, 3)
    v = _values(st, "v", s, pos[None].expand(S, L)).permute(0, 2, 1, 3)
    use = live[:, None] & (pos >= st["offsets"][..., None])
    u = st["u"][:, :, :L].expand(S, N, L, c["r"])
    return _attend(c, st["q"][:, :, None], k, v, u, st["b"], live[:, None], use)[:, :, 0].bfloat16()


def _chunk(st):
    c = st["case"]
    N, T, L = c["N"], c["T"], c["L"]
    pos = torch.arange(L, device=DEV)
    keep = pos[None] <= (L - T + torch.arange(T, device=DEV))[:, None]
    use = pos >= st["offsets"][..., None]
    u = st["u"].expand(1, N, L, c["r"])
    return _attend(c, st["q"][None], st["k_out"].float(), st["v_out"].float(), u, st["b"], keep[None],
                   use)[0].bfloat16()


def _cache(st):
    return {n: st[n] for n in ("k8", "v8", "k_scale", "v_scale")}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _handles(st):
    """What a program keeps beside its cache: the problem, views of the buffers and a workspace."""
    import lora_shared_kv_b200 as lrkv
    c = st["case"]
    h = {"lrkv": lrkv}
    h["prob"] = lrkv.make_problem(c["S"], c["N"], c["Hkv"] * c["G"], c["Hkv"], c["d"], c["r"],
                                  lrkv.BASE_LR_SHARED if c["shared_u"] else lrkv.BASE_SHARED)
    if c["paged"]:
        h["kv"] = lrkv.kv_view_quant_paged(st["k8"], st["v8"], st["k_scale"], st["v_scale"], st["table"])
    else:
        h["kv"] = lrkv.kv_view_quant_dense(st["k8"], st["v8"], st["k_scale"], st["v_scale"])
    need = lrkv.KV_QUANT_WORKSPACE_BYTES
    if "q" in st:
        h["u"] = lrkv.u_view(st["u"])
        if c["kind"] == "chunk":
            need = max(need, lrkv.lrkv_prefill_workspace_bytes(h["prob"], c["L"] - c["T"], c["T"]))
        else:
            need = max(need, lrkv.lrkv_decode_quant_workspace_bytes(h["prob"], st["max_len"]))
    if "k_new" in st:
        h["new"] = lrkv.kv_view_dense(st["k_new"].permute(0, 2, 1, 3), st["v_new"].permute(0, 2, 1, 3))
    if "k_out" in st:
        h["back"] = lrkv.kv_view_dense(st["k_out"], st["v_out"])
    h["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    return h


def _own(st):
    if "handles" not in st:
        st["handles"] = _handles(st)
    h, c = st["handles"], st["case"]
    lrkv = h["lrkv"]
    if c["kind"] in ("write", "step", "chunk"):
        lrkv.lrkv_quantize_kv(h["prob"], h["new"], c["T"], h["kv"], c["L"], st["first"], st["count"], h["ws"])
        if c["kind"] == "write":
            return _cache(st)
    if c["kind"] == "read":
        lrkv.lrkv_dequantize_kv(h["prob"], h["kv"], c["L"], c["T"], h["back"], st["first"], st["count"], h["ws"])
        return st["k_out"], st["v_out"]
    if c["kind"] == "chunk":
        lrkv.lrkv_dequantize_kv(h["prob"], h["kv"], c["L"], c["L"], h["back"], None, st["lens"], h["ws"])
        lrkv.lrkv_attn_prefill_chunk(h["prob"], st["q"], h["back"], 0, c["L"] - c["T"], c["T"], h["u"], st["b"],
                                     st["offsets"], st["out"], h["ws"])
        return {"out": st["out"], "k": st["k_out"], "v": st["v_out"], **_cache(st)}
    lrkv.lrkv_attn_decode_quant(h["prob"], st["q"], h["kv"], st["lens"], st["max_len"], h["u"], st["b"],
                                st["offsets"], st["out"], h["ws"])
    return {"out": st["out"], **_cache(st)} if c["kind"] == "step" else st["out"]


def run(state):
    if own:
        return _own(state)
    st = state
    kind = st["case"]["kind"]
    if kind in ("write", "step", "chunk"):
        _write(st, "k", st["k_new"])
        _write(st, "v", st["v_new"])
        if kind == "write":
            return _cache(st)
    if kind == "read":
        return _read(st, st["first"], st["count"], st["case"]["T"])
    if kind == "chunk":
        k, v = _read(st, torch.zeros_like(st["first"]), st["lens"], st["case"]["L"])
        return {"out": _chunk(st), "k": k, "v": v, **_cache(st)}
    return {"out": _decode(st), **_cache(st)} if kind == "step" else _decode(st)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    S, N, G, H, d, r, T = c["S"], c["N"], c["G"], c["Hkv"], c["d"], c["r"], c["T"]
    lens, first, count, offs = _plan(c)
    nbytes = flops = 0
    if c["kind"] in ("write", "step", "chunk"):
        nbytes += 2 * H * d * 3 * sum(count)                                          # bf16 in, codes out
        blocks = sum((f + n - 1) // BLOCK - f // BLOCK + 1 for f, n in zip(first, count) if n)
        nbytes += 2 * H * 4 * (blocks + sum(f % BLOCK > 0 for f, n in zip(first, count) if n)) + 8 * S
        flops += 2 * H * d * 2 * sum(count)
    if c["kind"] in ("read", "chunk"):
        rows = count if c["kind"] == "read" else lens
        nbytes += 2 * H * (d * 3 * sum(rows) + 4 * sum(-(-n // BLOCK) for n in rows)) + 8 * S
        flops += 2 * H * d * sum(rows)
    if c["kind"] in ("decode", "step"):
        nbytes += 2 * H * (d * sum(lens) + 4 * sum(-(-n // BLOCK) for n in lens))     # codes and scales
        used = [[max(0, n - a) for a in o] for n, o in zip(lens, offs)]
        nbytes += 2 * r * sum(max(x) if c["shared_u"] else sum(x) for x in used)      # U rows past the offsets
        nbytes += 2 * 2 * S * N * H * G * d + 2 * N * r * H * d + 4 * S * (N + 1)     # q, out, B, lengths, offsets
        flops += 4 * H * G * N * d * sum(lens) + 2 * H * G * r * sum(map(sum, used)) + 2 * S * N * H * G * r * d
    if c["kind"] == "chunk":
        L0 = c["L"] - T
        keys = T * L0 + T * (T + 1) // 2
        nbytes += 2 * H * d * 2 * c["L"] + 2 * r * sum(c["L"] - a for a in offs[0])
        nbytes += 2 * 2 * N * T * H * G * d + 2 * N * r * H * d
        flops += 2 * N * H * G * keys * (2 * d + r) + 2 * N * H * G * T * r * d
    if c["paged"]:
        nbytes += 4 * sum(-(-n // BLOCK) for n in (count if c["kind"] in ("write", "read") else lens))
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_table():
    """The 127 non-negative numbers of e4m3: (1 + m / 8) 2^(e - 7), and m / 8 * 2^-6 for e = 0."""
    vals = [m / 8 * 2.0 ** -6 for m in range(8)]
    vals += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]
    return torch.tensor(vals, dtype=torch.float64, device=DEV)


def _nearest(y, fmt):
    """y rounded to the format's numbers in fp64: nearest, ties to even, saturating."""
    if fmt == "int8":
        n = torch.floor(y)
        part = y - n
        up = (part > 0.5) | ((part == 0.5) & (torch.remainder(n, 2) == 1))
        return (n + up).clamp(-127, 127)
    tab = _e4m3_table()
    a = y.abs().clamp(max=E4M3_MAX)
    i = torch.searchsorted(tab, a, right=True).clamp(1, tab.numel() - 1) - 1
    lo, hi = tab[i], tab[i + 1]
    mid = (lo + hi) / 2
    up = (a > mid) | ((a == mid) & (i % 2 == 1))  # neighbours' codes alternate in parity
    return torch.where(torch.isnan(y), y, torch.copysign(torch.where(up, hi, lo), y))


def _logical(st, name):
    """Codes [S, Hkv, rows, d] and scales [S, Hkv, blocks] of a cache in logical order, in fp64."""
    codes, scale = st[name + "8"].to(torch.float32), st[name + "_scale"].double()
    if not st["case"]["paged"]:
        return codes.double(), scale
    t = st["table"].long()
    S, nb = t.shape
    y = codes[t.view(-1)].view(S, nb, *codes.shape[1:]).permute(0, 2, 1, 3, 4)
    return y.reshape(S, y.shape[1], nb * BLOCK, -1).double(), scale[t.view(-1)].view(S, nb, -1).permute(0, 2, 1)


def _two_to(lo, hi):
    """The powers of two 2^lo .. 2^hi, ascending."""
    return torch.tensor([2.0 ** k for k in range(lo, hi + 1)], dtype=torch.float64, device=DEV)


def _exact_write(st, name, lens, first, count):
    """The cache after the write: codes' values and scales, laid out as the state's, in fp64."""
    c = st["case"]
    y, s = (v.clone() for v in _logical(st, name))
    x = st[name + "_new"].double()
    top = E4M3_MAX if c["fmt"] == "e4m3" else 127.0
    for i in range(c["S"]):
        at, end = first[i], first[i] + count[i]
        while at < end:
            blk = at // BLOCK
            lo, hi = blk * BLOCK, min(end, (blk + 1) * BLOCK)
            new = x[i, at - first[i]:hi - first[i]].permute(1, 0, 2)                  # [Hkv, n, d]
            a = torch.where(torch.isfinite(new), new.abs(), 0.0).amax(dim=(1, 2)) / top
            twos = _two_to(-120, 130)
            if c["fmt"] == "e4m3":
                need = twos[torch.searchsorted(twos, a)]
            else:  # a rounded up to eight significant bits, on the grid of its binade
                grid = twos[(torch.searchsorted(twos, a, right=True) - 1).clamp_min(0)] / 128
                need = torch.ceil(a / grid) * grid
            need = need.clamp_min(SCALE_MIN)
            if at > lo:
                old = s[i, :, blk].clone()
                need = torch.maximum(need, old)
                y[i, :, lo:at] = _nearest(y[i, :, lo:at] * (old / need)[:, None, None] if c["fmt"] == "e4m3"
                                          else y[i, :, lo:at] * old[:, None, None] / need[:, None, None], c["fmt"])
            y[i, :, at:hi] = _nearest(new / need[:, None, None], c["fmt"])
            s[i, :, blk] = need
            at = hi
    return y, s


def _physical(st, y, s):
    if not st["case"]["paged"]:
        return y, s
    S, H, rows, d = y.shape
    nb = rows // BLOCK
    t = st["table"].long().view(-1)
    codes, scale = torch.empty((S * nb, H, BLOCK, d), dtype=torch.float64, device=DEV), None
    codes[t] = y.view(S, H, nb, BLOCK, d).permute(0, 2, 1, 3, 4).reshape(S * nb, H, BLOCK, d)
    scale = torch.empty((S * nb, H), dtype=torch.float64, device=DEV)
    scale[t] = s.permute(0, 2, 1).reshape(S * nb, H)
    return codes, scale


def _exact_rows(q, k, v, u, b, seen, a0):
    """One KV head: q [N, G, R, d], k, v [L, d], u [N or 1, L, r], b [N, r, d]; row R sees keys < seen[R]."""
    N, G, R, d = q.shape
    L = k.shape[0]
    pos = torch.arange(L, device=DEV)
    out = torch.empty((N, G, R, d), dtype=torch.float64, device=DEV)
    for n in range(N):
        w = (q[n].reshape(G * R, d) @ k.T).view(G, R, L) * d ** -0.5
        w = w.masked_fill(pos >= seen[:, None], -math.inf).softmax(-1)
        val = v + (u[n % u.shape[0]] * (pos >= a0[n])[:, None]) @ b[n]
        out[n] = w @ val
    return out


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    lens, first, count, offs = _plan(c)
    H, G, d, N, r = c["Hkv"], c["G"], c["d"], c["N"], c["r"]
    log = {n: _logical(st, n) for n in ("k", "v")}
    done = {}
    if c["kind"] in ("write", "step", "chunk"):
        if sum(-(-n // BLOCK) + 1 for n in count) > 4000:
            return None  # block by block this would take too long
        for n in ("k", "v"):
            log[n] = _exact_write(st, n, lens, first, count)
            done[n + "8"], done[n + "_scale"] = _physical(st, *log[n])
            if c["fmt"] == "int8":
                done[n + "8"] = None  # whole numbers: compared as they are
        if c["kind"] == "write":
            return {k: done[k] for k in ("k8", "v8", "k_scale", "v_scale")}
    val = {}
    for n in ("k", "v"):
        y, s = log[n]
        val[n] = y * s.repeat_interleave(BLOCK, dim=2)[:, :, :y.shape[2], None]
    if c["kind"] == "read":
        res = []
        for n in ("k", "v"):
            out = st[n + "_out"].double()
            for i in range(c["S"]):
                out[i, :, :count[i]] = val[n][i, :, first[i]:first[i] + count[i]]
            res.append(out)
        return tuple(res)
    q, u, b = st["q"].double(), st["u"].double(), st["b"].double().view(N, r, H, d)
    if c["kind"] == "chunk":
        # the chunk attends to the rows as bf16 holds them
        held = {n: val[n][:, :, :c["L"]].bfloat16().double() for n in ("k", "v")}
        seen = c["L"] - c["T"] + 1 + torch.arange(c["T"], device=DEV)
        out = torch.empty(q.shape, dtype=torch.float64, device=DEV)
        for g in range(H):
            o = _exact_rows(q[:, :, g * G:(g + 1) * G].permute(0, 2, 1, 3), held["k"][0, g], held["v"][0, g], u[0],
                            b[:, :, g], seen, offs[0])
            out[:, :, g * G:(g + 1) * G] = o.permute(0, 2, 1, 3)
        return {"out": out, "k": val["k"][:, :, :c["L"]], "v": val["v"][:, :, :c["L"]], **done}
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    for i in range(c["S"]):
        if lens[i] == 0:
            continue
        seen = torch.tensor([lens[i]], device=DEV)
        for g in range(H):
            o = _exact_rows(q[i, :, g * G:(g + 1) * G, None], val["k"][i, g, :lens[i]], val["v"][i, g, :lens[i]],
                            u[i, :, :lens[i]], b[:, :, g], seen, offs[i])
            out[i, :, g * G:(g + 1) * G] = o[:, :, 0]
    return {"out": out, **done} if c["kind"] == "step" else out
