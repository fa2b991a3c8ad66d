"""The 8-bit cache on the GPU: every bf16 magnitude's scale and code, the bound of large scores as derived, and
shapes whose U tiles leave the least shared memory."""

import numpy as np
import pytest
import torch

import lora_shared_kv_b200 as lrkv
from oracle import kvq_oracle as kvq
from test_gpu_quant import DEV, DecodeCase, _flags_ws, _numbers, DTYPE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_every_finite_bf16_magnitude(fmt):
    """32,640 blocks of one row, one for each finite magnitude a: a, -a and fractions of it, some of them ties."""
    a = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    S, d = a.numel(), 64
    part = torch.cat([torch.tensor([1.0, -1.0]), torch.arange(31) / 32, -(torch.arange(31) + 0.5) / 127])
    x = (a.double()[:, None] * part.double()).to(torch.bfloat16).view(S, 1, 1, d)
    assert torch.isfinite(x).all() and torch.equal(x[:, 0, 0, 0], a)
    codes = torch.zeros((S, 1, 64, d), dtype=torch.uint8, device=DEV).view(DTYPE[fmt])
    scale = torch.full((S, 1, 1), float("nan"), device=DEV)
    other, spare = codes.clone(), scale.clone()
    prob = lrkv.make_problem(S, 1, 1, 1, d, 8)
    ws = _flags_ws()
    lrkv.lrkv_quantize_kv(prob, lrkv.kv_view_dense(x.to(DEV), x.to(DEV)), 1,
                          lrkv.kv_view_quant_dense(codes, other, scale, spare), 64, None, None, ws)
    assert lrkv.lrkv_query_device_status(ws)[0] == "LRKV_OK"
    want = np.array([kvq.scale_for(float(v), fmt) for v in a.double()])
    assert np.array_equal(scale.double().cpu().numpy().reshape(-1), want)
    got = _numbers(codes)[:, 0]
    assert np.array_equal(got[:, 0], kvq.nearest(x.double().numpy()[:, 0, 0] / want[:, None], fmt))
    assert not got[:, 1:].any()
    assert torch.equal(codes.view(torch.uint8), other.view(torch.uint8)) and torch.equal(scale, spare)


def test_large_scores_within_the_derived_bound():
    # sum |q k| scale is about 217: 4 * 128 * 217 * 2^-24 = 27 * 2^-12 (see test_gpu_quant)
    c = DecodeCase("large", "int8", 1, 2, 4, 1, 128, 16, 300, 0, [0, 150], [300], q_std=30.0)
    c.check(c.run(), "large", weight=27.0)


TIGHT = [  # S, N, G, Hkv, d, r, L, mode, offsets, lens: up to 16 U tiles of 4 KB a stage
    (1, 16, 2, 1, 128, 32, 1100, 0, list(range(0, 1040, 65)), [1100]),       # 32 rows, one item's 16 agents
    (2, 16, 3, 1, 128, 32, 700, 0, [(41 * i) % 710 for i in range(32)], [700, 333]),   # 48 rows: two groups of 24
    (1, 16, 8, 2, 128, 32, 500, 0, list(range(0, 512, 32)), [500]),          # 128 rows: four groups of 32
    (2, 13, 1, 3, 128, 32, 900, 0, [(67 * i) % 910 for i in range(26)], [900, 65]),    # 13 rows
    (160, 16, 1, 1, 128, 32, 400, 0, [(67 * i) % 410 for i in range(16 * 160)], [1 + (37 * i) % 400 for i in range(160)]),
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("shape", TIGHT, ids=[f"S{s[0]}N{s[1]}G{s[2]}" for s in TIGHT])
def test_the_largest_u_tiles(shape, fmt):
    c = DecodeCase(shape, fmt, *shape)
    c.check(c.run(), str(shape))
