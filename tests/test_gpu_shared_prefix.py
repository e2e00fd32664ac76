"""Decode of a batch with a shared prefix against the 64-bit definition."""
import math

import pytest
import torch

from rows_reference import attend64, check_rows, gather_pages, generator, randn, random_pool

pytestmark = pytest.mark.gpu


def run_paged(fd, lens, skip, Hq, Hkv, d, seed, **kw):
    """lens: all tokens of every sequence, the first skip * 64 shared."""
    g = generator(seed)
    kp, vp, table, pool = random_pool([max(n, skip * 64) for n in lens], Hkv, d, g, skip=skip)
    for b, n in enumerate(lens):  # nothing behind a sequence's end in its own pages
        if n <= skip * 64:
            table[b, skip:] = -1
    q = randn(g, len(lens), Hq, d)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    prefix = table[0, :skip].clone()
    rows = table.clone()
    rows[:, :skip] = -7  # not read
    out, lse = fd.fd_decode_paged_shared_prefix(q, kp, vp, prefix, rows, pool, sl, **kw)
    for b, n in enumerate(lens):
        k, v = gather_pages(kp, table[b], n), gather_pages(vp, table[b], n)
        check_rows(out[b:b + 1], lse[b:b + 1], attend64(q[b:b + 1], k, v, torch.tensor([n]), 1 / math.sqrt(d)),
                   f"sequence {b} of {n} tokens")
    assert fd.fd_device_status(clear=True) == fd.FD_OK
    return q, kp, vp, prefix, rows, table, pool, sl, out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_paged(fd, G, d):
    run_paged(fd, [700, 641, 640, 1500, 900], 10, 2 * G, 2, d, seed=G)


@pytest.mark.parametrize("B", [1, 2, 16, 31, 33, 70, 130])
def test_batch_sizes(fd, B):
    lens = [64 * 5 + (37 * b) % 300 for b in range(B)]
    run_paged(fd, lens, 5, 8, 1, 128, seed=B)


@pytest.mark.parametrize("num_splits", [0, 1, 2, 9])
def test_splits_and_float32(fd, num_splits):
    run_paged(fd, [3000, 2560, 4000], 40, 8, 2, 128, seed=1, num_splits=num_splits, out_dtype="f32")


def test_sequences_shorter_than_the_prefix(fd):
    # padded rows of a batch (length 0) and sequences that end inside the shared tokens
    *_, out, lse = run_paged(fd, [0, 1, 63, 64, 100, 639, 640, 641, 0], 10, 8, 2, 128, seed=2)
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[8]))


def test_no_prefix_and_nothing_but_prefix(fd):
    run_paged(fd, [100, 1, 0, 333], 0, 4, 2, 64, seed=3)
    run_paged(fd, [640] * 4, 10, 4, 2, 64, seed=4)


def test_is_the_paged_decode_of_the_whole_sequences(fd):
    q, kp, vp, prefix, rows, table, pool, sl, out, lse = run_paged(fd, [5000, 4500, 4100], 64, 8, 2, 128, seed=5)
    want, wlse = fd.fd_decode_paged(q, kp, vp, table, pool, sl)
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -7
    assert (lse - wlse).abs().max() < 1e-4


def test_bad_shared_page_is_skipped_and_reported(fd):
    g = generator(6)
    lens, skip = [400, 500], 4
    kp, vp, table, pool = random_pool(lens, 2, 128, g, skip=skip)
    q = randn(g, 2, 8, 128)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    prefix = table[0, :skip].clone()
    prefix[1] = pool
    out, lse = fd.fd_decode_paged_shared_prefix(q, kp, vp, prefix, table, pool, sl)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_BAD_PAGE_TABLE
    for b, n in enumerate(lens):
        k, v = gather_pages(kp, table[b], n), gather_pages(vp, table[b], n)
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep[64:128] = False
        check_rows(out[b:b + 1], lse[b:b + 1],
                   attend64(q[b:b + 1], k[keep], v[keep], torch.tensor([n - 64]), 1 / math.sqrt(128)))


@pytest.mark.parametrize("P", [1, 63, 64, 1000, 4097])
@pytest.mark.parametrize("G,d", [(1, 128), (4, 128), (8, 64)])
def test_dense(fd, P, G, d):
    g = generator(P)
    B, Hkv, L = 5, 2, 300
    q = randn(g, B, Hkv * G, d)
    kp, vp = randn(g, Hkv, P, d), randn(g, Hkv, P, d)
    k, v = randn(g, B, Hkv, L, d), randn(g, B, Hkv, L, d)
    lens = [0, 1, 64, 299, 300]
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = float("nan"), float("nan")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = fd.fd_decode_dense_shared_prefix(q, kp, vp, k, v, sl)
    for b, n in enumerate(lens):
        kk = torch.cat([kp, k[b, :, :n]], dim=1).transpose(0, 1)
        vv = torch.cat([vp, v[b, :, :n]], dim=1).transpose(0, 1)
        check_rows(out[b:b + 1], lse[b:b + 1],
                   attend64(q[b:b + 1], kk, vv, torch.tensor([P + n]), 1 / math.sqrt(d)), f"sequence {b}")
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_dense_without_prefix_or_own_tokens(fd):
    g = generator(8)
    q = randn(g, 3, 4, 64)
    k, v = randn(g, 3, 2, 100, 64), randn(g, 3, 2, 100, 64)
    out, lse = fd.fd_decode_dense_shared_prefix(q, k[0, :, :0].contiguous(), v[0, :, :0].contiguous(), k, v)
    want, wlse = fd.fd_decode_dense(q, k, v)
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -7 and (lse - wlse).abs().max() < 1e-5
    out, lse = fd.fd_decode_dense_shared_prefix(q, k[0].contiguous(), v[0].contiguous(), k[:, :, :0].contiguous(),
                                                v[:, :, :0].contiguous())
    for b in range(3):
        check_rows(out[b:b + 1], lse[b:b + 1],
                   attend64(q[b:b + 1], k[0].transpose(0, 1), v[0].transpose(0, 1), torch.tensor([100]), 1 / 8))


def test_long_prefix_large_batch_sampled(fd):
    g = generator(9)
    B, Hq, Hkv, d, skip = 60, 64, 8, 128, 300
    lens = [skip * 64 + (b * 31) % 500 for b in range(B)]
    kp, vp, table, pool = random_pool(lens, Hkv, d, g, skip=skip)
    q = randn(g, B, Hq, d)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = fd.fd_decode_paged_shared_prefix(q, kp, vp, table[0, :skip].clone(), table, pool, sl)
    for b in (0, 15, 16, 17, 31, 59):
        k, v = gather_pages(kp, table[b], lens[b]), gather_pages(vp, table[b], lens[b])
        check_rows(out[b:b + 1], lse[b:b + 1], attend64(q[b:b + 1], k, v, torch.tensor([lens[b]]), 1 / math.sqrt(d)))


def test_two_graphs_share_a_workspace(fd):
    q, kp, vp, prefix, rows, table, pool, sl, want, wlse = run_paged(fd, [900, 1000, 641], 10, 8, 2, 128, seed=10)
    n = fd.fd_shared_prefix_workspace_size(3, 8, 2, 640, (rows.shape[1] - 10) * 64, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for i in range(2):
        out, lse = torch.empty_like(want), torch.empty_like(wlse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fd.fd_decode_paged_shared_prefix(q, kp, vp, prefix, rows, pool, sl, out=out, lse=lse, workspace=ws)
        outs.append((out, lse))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out, want) and torch.equal(lse, wlse)
