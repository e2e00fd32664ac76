"""Differential calls whose keys are cut into many parts: lists longer than a warp of the merge holds at once, by one
warp a map and by four."""
import math

import pytest
import torch

from diff_reference import check_diff, diff64, generator, ints, limits, rand, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("splits", [9, 33, 40, 140, 200])
def test_decode(fd, splits, d, norm):
    """Few rows, lists of up to 200 records, some of them empty."""
    g = generator(splits + d)
    lens = [13000, 0, 700, 64 * 37, 1, 64 * 200]
    B, Hq, Hkv, L = len(lens), 4, 2, 13000
    q, k, v = randn(g, B, Hq, d), randn(g, B, Hkv, L, d), randn(g, B, Hkv, L, d)
    lam, w = rand(g, 0.1, 0.6, B, Hq), rand(g, 0.2, 1.5, d) if norm else None
    assert fd.fd_num_splits_diff(B, Hq, Hkv, L, d, splits, True) == splits
    out, lse = fd.fd_decode_dense_diff(q, k, v, lam, ints(lens), norm_weight=w, num_splits=splits, out_dtype="f32")
    for b, n in enumerate(lens):
        ref = diff64(q[b:b + 1], k[b, :, :n].transpose(0, 1), v[b, :, :n].transpose(0, 1), lam[b:b + 1], limits(1, n),
                     1 / math.sqrt(d // 2), w, rounding=2.0 ** -16)
        check_diff(out[b:b + 1], lse[b:b + 1], ref, str(b))
    assert fd.fd_device_status(clear=True) == fd.FD_OK


@pytest.mark.parametrize("splits", [8, 9, 16, 40])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 1, 64), (16, 4, 128)])
def test_decode_of_many_rows(fd, Hq, Hkv, d, splits):
    """4096 rows and more: one warp a map, more than 8 records."""
    B, L = 4096 // Hq, 2600
    g = generator(splits + Hq)
    lens = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[:3] = ints([L, 0, 1])
    q, k, v = randn(g, B, Hq, d), randn(g, B, Hkv, L, d), randn(g, B, Hkv, L, d)
    lam = rand(g, 0.1, 0.6, Hq)
    out, lse = fd.fd_decode_dense_diff(q, k, v, lam, lens, num_splits=splits, out_dtype="f32")
    for b in [0, 1, 2, *range(3, B, 37), B - 1]:
        n = int(lens[b])
        ref = diff64(q[b:b + 1], k[b, :, :n].transpose(0, 1), v[b, :, :n].transpose(0, 1), lam, limits(1, n),
                     1 / math.sqrt(d // 2), rounding=2.0 ** -16)
        check_diff(out[b:b + 1], lse[b:b + 1], ref, str(b))
    assert fd.fd_device_status(clear=True) == fd.FD_OK


@pytest.mark.parametrize("T,Hq,Hkv,d", [(70, 4, 2, 128), (1100, 4, 1, 64)])
def test_prompts(fd, T, Hq, Hkv, d):
    """40 parts of one sequence, of few rows and of more than 4096."""
    L, splits = 128 * 41 + 5, 40
    g = generator(T)
    q, k, v = randn(g, T, Hq, d), randn(g, L, Hkv, d), randn(g, L, Hkv, d)
    lam, w = rand(g, 0.1, 0.6, Hq), rand(g, 0.2, 1.5, d)
    assert fd.fd_prefill_diff_num_splits(1, T, Hq, Hkv, L, d, splits) == splits
    out, lse = fd.fd_prefill_packed_diff(q, k, v, lam, ints([0, T]), ints([0, L]), norm_weight=w, num_splits=splits,
                                         out_dtype="f32")
    check_diff(out, lse, diff64(q, k, v, lam, limits(T, L), 1 / math.sqrt(d // 2), w, rounding=2.0 ** -16))
    assert fd.fd_device_status(clear=True) == fd.FD_OK
