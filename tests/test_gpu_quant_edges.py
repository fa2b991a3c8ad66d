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
