"""Weights that enter the product with V in two bf16 terms: the float32 results
of every prompt and shared-prefix call.

hi = bf16(w) is off by at most 2^-8 w, lo = bf16(w - hi) by at most 2^-8 of
that: 2^-16 w together (w - hi is exact in binary32).  So the bound of
rows_reference with 2^-16 in place of 2^-8.
"""
import math

import pytest
import torch

from rows_reference import attend64, check_rows, gather_pages, generator, limits, offsets, randn, random_pool

pytestmark = pytest.mark.gpu


def fine64(q, k, v, limit, scale):
    out, lse, bound, lse_bound = attend64(q, k, v, limit, scale)
    weight = attend64(q, k, v.abs(), limit, scale)[0]  # sum_j w_j |v_j|
    return out, lse, bound - (2.0 ** -8 - 2.0 ** -16) * weight, lse_bound


def check_packed(fd, lens_q, lens_k, Hq, Hkv, d, causal, num_splits, seed):
    g = generator(seed)
    q, k, v = randn(g, sum(lens_q), Hq, d), randn(g, sum(lens_k), Hkv, d), randn(g, sum(lens_k), Hkv, d)
    out, lse = fd.fd_prefill_packed(q, k, v, offsets(lens_q), offsets(lens_k), causal=causal, num_splits=num_splits,
                                    out_dtype="f32")
    a = b = 0
    for n, m in zip(lens_q, lens_k):
        check_rows(out[a:a + n], lse[a:a + n],
                   fine64(q[a:a + n], k[b:b + m], v[b:b + m], limits(n, m, causal), 1 / math.sqrt(d)), f"{n} on {m}")
        a, b = a + n, b + m
    assert fd.fd_device_status(clear=True) == fd.FD_OK


@pytest.mark.parametrize("num_splits", [0, 1, 3])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,d", [(1, 64), (1, 128), (3, 128), (4, 64), (8, 128)])
def test_packed(fd, G, d, causal, num_splits):
    lens = [1, 0, 63, 64, 65, 127, 128, 129, 300, 2, 257, 1000]
    check_packed(fd, lens, lens, 2 * G, 2, d, causal, num_splits, seed=G)


@pytest.mark.parametrize("num_splits", [0, 1, 3])
@pytest.mark.parametrize("G,d", [(1, 64), (4, 128), (7, 128), (8, 64)])
def test_packed_few_queries(fd, G, d, num_splits):
    check_packed(fd, [1, 9, 16, 3], [500, 9, 1300, 128], 2 * G, 2, d, True, num_splits, seed=G)


@pytest.mark.parametrize("num_splits", [0, 1, 4])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [8, 3, 16, 0], [200, 64, 1, 130]], ids=str)
@pytest.mark.parametrize("G,d", [(1, 128), (4, 64), (8, 128)])
def test_paged(fd, new, G, d, num_splits):
    g = generator(G)
    total = [n + c for n, c in zip(new, (0, 1000, 129, 63))]
    kp, vp, table, pool = random_pool(total, 2, d, g)
    q = randn(g, sum(new), 2 * G, d)
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    out, lse = fd.fd_prefill_paged(q, kp, vp, table, pool, offsets(new), lens, num_splits=num_splits, out_dtype="f32")
    a = 0
    for i, (n, L) in enumerate(zip(new, total)):
        k, v = gather_pages(kp, table[i], L), gather_pages(vp, table[i], L)
        check_rows(out[a:a + n], lse[a:a + n], fine64(q[a:a + n], k, v, limits(n, L, True), 1 / math.sqrt(d)))
        a += n
    assert fd.fd_device_status(clear=True) == fd.FD_OK


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("B,G,d", [(5, 4, 128), (16, 8, 128), (5, 1, 64), (40, 4, 64), (130, 1, 128)])
def test_shared_prefix(fd, B, G, d, paged):
    g = generator(B)
    skip, Hkv = 11, 2
    own = [(37 * b) % 300 for b in range(B)]
    q = randn(g, B, Hkv * G, d)
    if paged:
        lens = [skip * 64 + n for n in own]
        kp, vp, table, pool = random_pool(lens, Hkv, d, g, skip=skip)
        out, lse = fd.fd_decode_paged_shared_prefix(q, kp, vp, table[0, :skip].clone(), table, pool,
                                                    torch.tensor(lens, dtype=torch.int32, device="cuda"), out_dtype="f32")
        tokens = [(gather_pages(kp, table[b], n), gather_pages(vp, table[b], n)) for b, n in enumerate(lens)]
    else:
        kp, vp = randn(g, Hkv, 700, d), randn(g, Hkv, 700, d)
        k, v = randn(g, B, Hkv, 300, d), randn(g, B, Hkv, 300, d)
        out, lse = fd.fd_decode_dense_shared_prefix(q, kp, vp, k, v, torch.tensor(own, dtype=torch.int32, device="cuda"),
                                                    out_dtype="f32")
        tokens = [(torch.cat([kp, k[b, :, :n]], 1).transpose(0, 1), torch.cat([vp, v[b, :, :n]], 1).transpose(0, 1))
                  for b, n in enumerate(own)]
    for b, (k, v) in enumerate(tokens):
        check_rows(out[b:b + 1], lse[b:b + 1],
                   fine64(q[b:b + 1], k, v, torch.tensor([k.shape[0]]), 1 / math.sqrt(d)), f"sequence {b}")
    assert fd.fd_device_status(clear=True) == fd.FD_OK


@pytest.mark.parametrize("std,scale", [(30.0, 1.0), (1e-3, 0.1), (1.0, 1e-6), (8.0, 0.125)])
@pytest.mark.parametrize("T", [20, 300])
def test_extreme_scores(fd, T, std, scale):
    # one key takes nearly all the weight, or all weigh the same: the outputs themselves are checked
    g = generator(11)
    q = (torch.randn((T, 4, 64), generator=g, device="cuda") * std).to(torch.bfloat16)
    k = (torch.randn((T, 2, 64), generator=g, device="cuda") * std).to(torch.bfloat16)
    v = randn(g, T, 2, 64)
    out, lse = fd.fd_prefill_packed(q, k, v, offsets([T]), scale=scale, out_dtype="f32")
    check_rows(out, lse, fine64(q, k, v, limits(T, T, True), scale))
    # tighter where scores are large: a key's weight is off by its own score's error, not the largest one's
    s = torch.einsum("thd,lhd->htl", q.double(), k.double().repeat_interleave(2, 1)) * scale
    es = 64 * 2.0 ** -23 * torch.einsum("thd,lhd->htl", q.double().abs(), k.double().abs().repeat_interleave(2, 1)) * scale
    hidden = torch.arange(T, device="cuda")[None, :] > torch.arange(T, device="cuda")[:, None]
    w = torch.softmax(s.masked_fill(hidden[None], float("-inf")), -1)
    vv = v.double().repeat_interleave(2, 1)
    want = torch.einsum("htl,lhd->thd", w, vv)
    # every weight w_j may be off by a factor e^(+-2 es_j), the sum by the weighted mean of those, and the product by
    # 2^-16 and n + 1 roundings
    err = torch.expm1(2 * es)
    mean = (w * err).sum(-1, keepdim=True)
    bound = torch.einsum("htl,lhd->thd", w * (err + mean) * (1 + mean), vv.abs())
    bound += torch.einsum("htl,lhd->thd", w, vv.abs()) * (2.0 ** -16 + 2.0 ** -20 + T * 2.0 ** -22)
    assert ((out.double() - want).abs() <= bound * (1 + mean.max()) + 2.0 ** -23 * want.abs() + 1e-30).all()


def test_single_tokens_are_the_paged_decode(fd):
    # both passes hold 2^-16 weights: float32 results differ by twice the bound
    g = generator(5)
    lens = [1, 63, 64, 65, 1000, 5000]
    kp, vp, table, pool = random_pool(lens, 2, 128, g)
    q = randn(g, len(lens), 8, 128)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = fd.fd_prefill_paged(q, kp, vp, table, pool, offsets([1] * len(lens)), sl, out_dtype="f32")
    want, wlse = fd.fd_decode_paged(q, kp, vp, table, pool, sl, out_dtype="f32")
    for b, n in enumerate(lens):
        k, v = gather_pages(kp, table[b], n), gather_pages(vp, table[b], n)
        _, _, bound, lse_bound = fine64(q[b:b + 1], k, v, torch.tensor([n]), 1 / math.sqrt(128))
        assert ((out[b] - want[b]).abs() <= 2 * bound[0] + 2.0 ** -22 * want[b].abs()).all()
        assert ((lse[b] - wlse[b]).abs() <= 2 * lse_bound[0]).all()
