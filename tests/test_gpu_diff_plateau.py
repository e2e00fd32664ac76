"""Scores that rise by a moderate amount over very many keys: it is a row's sum of weights, not one score, that
passes what a single pass holds."""
import math

import pytest
import torch

from diff_reference import check_diff, diff64, generator, ints, limits, rand, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rise", [14.0, 17.5, 18.5, 22.0, 27.5, 28.5])
def test_a_plateau_over_16k_keys(fd, rise, dtype, splits):
    """2^40 is reached by 2^14 keys at 26 ln 2 = 18.02 above the first, by one at 40 ln 2 = 27.7.  The first 64
    keys score 0 in the first map, the others `rise` plus a spread; the second map is an ordinary one."""
    g = generator(int(10 * rise))
    T, L, Hq, Hkv, d = 40, (1 << 14) + 64, 4, 2, 64
    q, k, v = randn(g, T, Hq, d), randn(g, L, Hkv, d), randn(g, L, Hkv, d)
    scale = 1 / math.sqrt(d // 2)
    q[..., :32], k[..., :32] = 0.25 * q[..., :32], 0.25 * k[..., :32]
    q[..., 0] = 1.0
    k[:64, :, :32] = 0.0
    k[64:, :, 0] = rise / scale
    lam, w = rand(g, 0.1, 0.6, Hq), rand(g, 0.2, 1.5, d)
    out, lse = fd.fd_prefill_packed_diff(q, k, v, lam, ints([0, T]), ints([0, L]), num_splits=splits, out_dtype=dtype)
    # (the norm would say nothing: what is left of 16K values is as small as the maps' errors)
    check_diff(out, lse, diff64(q, k, v, lam, limits(T, L), scale, rounding=2.0 ** -8 if dtype == "bf16" else 2.0 ** -16))
    assert fd.fd_device_status(clear=True) == fd.FD_OK
