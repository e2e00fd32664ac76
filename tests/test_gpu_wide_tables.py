"""Page tables far wider than their sequences: the parts that a plan leaves
without keys write no output of their own, and nothing of what the workspace
held before gets into a result."""
import math

import pytest
import torch

from rows_reference import attend64, check_rows, gather_pages, generator, limits, offsets, randn, random_pool

pytestmark = pytest.mark.gpu


def widen(table, room):
    wide = torch.full((table.shape[0], room), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    return wide


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx,Hq,Hkv,d", [([16, 3, 0, 1], [1000, 0, 70, 2000], 8, 2, 128),
                                              ([1] * 8, [2000] * 8, 32, 8, 128), ([100, 90], [500, 40], 8, 2, 64),
                                              ([300], [4000], 6, 2, 128)], ids=str)
def test_paged_prompts(fd, new, ctx, Hq, Hkv, d, causal):
    g = generator(len(new))
    total = [n + c for n, c in zip(new, ctx)]
    kp, vp, table, pool = random_pool(total, Hkv, d, g)
    wide = widen(table, 1024)
    q = randn(g, sum(new), Hq, d)
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    S = fd.fd_prefill_num_splits(len(new), sum(new), Hq, Hkv, 1024 * 64, d)
    assert S > 2
    ws = torch.full((fd.fd_prefill_workspace_size(len(new), sum(new), Hq, Hkv, 1024 * 64, d),), 255, dtype=torch.uint8,
                    device="cuda")
    out, lse = fd.fd_prefill_paged(q, kp, vp, wide, pool, offsets(new), lens, causal=causal, workspace=ws)
    a = 0
    for i, (n, L) in enumerate(zip(new, total)):
        k, v = gather_pages(kp, table[i], L), gather_pages(vp, table[i], L)
        check_rows(out[a:a + n], lse[a:a + n], attend64(q[a:a + n], k, v, limits(n, L, causal), 1 / math.sqrt(d)),
                   f"sequence {i}")
        chunk = max(512, -(-(-(-L // 128)) // S) * 128)
        if (S - 1) * chunk >= L:  # the last part has no keys: its outputs are as the workspace was
            o = ws[:sum(new) * Hq * S * d * 4].view(torch.int32).view(sum(new), Hq, S, d)
            assert torch.all(o[a:a + n, :, -1] == -1)
        a += n
    assert fd.fd_device_status(clear=True) == fd.FD_OK


@pytest.mark.parametrize("lens", [[700, 641, 640, 5000, 0, 12], [640] * 40, [641 + 40 * b for b in range(40)]], ids=str)
@pytest.mark.parametrize("G,d", [(1, 128), (4, 64), (8, 128)])
def test_shared_prefix(fd, lens, G, d):
    g = generator(G)
    skip, Hkv, B = 10, 2, len(lens)
    kp, vp, table, pool = random_pool([max(n, skip * 64) for n in lens], Hkv, d, g, skip=skip)
    wide = widen(table, skip + 2000)
    q = randn(g, B, Hkv * G, d)
    ws = torch.full((fd.fd_shared_prefix_workspace_size(B, Hkv * G, Hkv, skip * 64, 2000 * 64, d),), 255,
                    dtype=torch.uint8, device="cuda")
    out, lse = fd.fd_decode_paged_shared_prefix(q, kp, vp, table[0, :skip].clone(), wide, pool,
                                                torch.tensor(lens, dtype=torch.int32, device="cuda"), workspace=ws)
    for b, n in enumerate(lens):
        k, v = gather_pages(kp, table[b], n), gather_pages(vp, table[b], n)
        check_rows(out[b:b + 1], lse[b:b + 1], attend64(q[b:b + 1], k, v, torch.tensor([n]), 1 / math.sqrt(d)),
                   f"sequence {b} of {n} tokens")
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_a_long_run_of_empty_parts_is_no_time_out(fd):
    # 8 heads x 65535 parts, one of each with keys: some 3400 empty parts in a row on every SM take about 3 ms.  The
    # warps that wait for work meanwhile hear from the copy warp often enough for a limit of 1 ms.
    g = generator(3)
    T, H, d = 4, 8, 64
    q, k, v = randn(g, T, H, d), randn(g, T, H, d), randn(g, T, H, d)
    cu = offsets([T])
    ws = torch.empty(fd.fd_prefill_workspace_size(1, T, H, H, T, d, 65535), dtype=torch.uint8, device="cuda")
    fd.fd_prefill_packed(q, k, v, cu, num_splits=65535, workspace=ws)
    assert fd.fd_device_status(clear=True) == fd.FD_OK
    try:
        fd.fd_debug_inject_wait_timeout(1_000_000, -1)
        out, lse = fd.fd_prefill_packed(q, k, v, cu, num_splits=65535, workspace=ws)
        assert fd.fd_device_status(clear=True) == fd.FD_OK
    finally:
        fd.fd_debug_inject_wait_timeout(0, -1)
    check_rows(out, lse, attend64(q, k, v, limits(T, T, True), 1 / math.sqrt(d)))
