"""Page assignment and cache append, and a serving run of all prompt calls."""
import math
import random

import pytest
import torch

from rows_reference import attend64, check_rows, gather_pages, generator, limits, randn

pytestmark = pytest.mark.gpu


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def assign_plain(table, cached, new, free, head, total):
    """Lists in, lists out: the definition, one token at a time."""
    table = [list(r) for r in table]
    lens, cu, slots = [], [0], []
    for b, (c, n) in enumerate(zip(cached, new)):
        for j in range(-(-c // 64), -(-(c + n) // 64)):
            table[b][j] = free[head]
            head += 1
        for pos in range(c, c + n):
            slots.append(table[b][pos // 64] * 64 + pos % 64)
        lens.append(c + n)
        cu.append(cu[-1] + n)
    return table, lens, cu, slots + [-1] * (total - len(slots)), head


def problem(B, ctx, most, seed, wide=None, spare=5):
    r = random.Random(seed)
    cached = [r.randint(0, ctx) for _ in range(B)]
    new = [r.randint(0, most) for _ in range(B)]
    need = [-(-(c + n) // 64) for c, n in zip(cached, new)]
    wide = wide or max(1, max(need, default=1))
    ids = list(range(sum(need) + spare))
    r.shuffle(ids)
    table, at = [], 0
    for c in cached:
        n = -(-c // 64)
        table.append(ids[at:at + n] + [-1] * (wide - n))
        at += n
    return cached, new, table, ids[at:]


@pytest.mark.parametrize("B,ctx,most", [(1, 0, 1), (1, 0, 300), (3, 200, 130), (70, 500, 1), (256, 3000, 1),
                                        (1023, 100, 70), (1025, 100, 3), (2500, 90, 20), (40, 1000, 3000), (1030, 70, 601),
                                        (3100, 10, 3)])
@pytest.mark.parametrize("pad", [0, 37])
def test_assign(fd, B, ctx, most, pad):
    cached, new, table, free = problem(B, ctx, most, seed=B + most)
    total = sum(new) + pad
    want = assign_plain(table, cached, new, [0, 0] + free, 2, total)
    t = ints(table)
    lens, cu, slots, head = fd.fd_assign_pages(t, ints(cached), ints(new), ints([0, 0] + free), total,
                                               free_head=ints([2]))
    assert t.tolist() == want[0]
    assert lens.tolist() == want[1] and cu.tolist() == want[2] and slots.tolist() == want[3]
    assert head.tolist() == [want[4]]
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_assign_in_place_over_steps(fd):
    # a decode loop: lengths and the head of the free list updated where they are
    B = 300
    cached, _, table, free = problem(B, 130, 0, seed=1, wide=8, spare=B * 6)
    t, lens, head, one = ints(table), ints(cached), ints([0]), ints([1] * B)
    for step in range(130):
        want = assign_plain(table, cached, [1] * B, free, int(head.item()), B)
        _, _, slots, _ = fd.fd_assign_pages(t, lens, one, ints(free), B, free_head=head, seq_lens=lens,
                                            free_head_out=head)
        table, cached = want[0], want[1]
        assert slots.tolist() == want[3] and lens.tolist() == cached and head.tolist() == [want[4]]
    assert t.tolist() == table


@pytest.mark.parametrize("B,ctx,most", [(300, 100, 200), (1500, 50, 30), (3, 4000, 9000), (2100, 0, 9),
                                        (1500, 50, 60), (4, 100, 20000), (2100, 1000, 40)])
def test_assign_in_place_with_many_tokens(fd, B, ctx, most):
    # beyond what one block does alone: a cluster for the table, the whole GPU for the slots
    cached, new, table, free = problem(B, ctx, most, seed=B, spare=9)
    total = sum(new) + 13
    want = assign_plain(table, cached, new, free, 0, total)
    t, lens, head = ints(table), ints(cached), ints([0])
    _, cu, slots, _ = fd.fd_assign_pages(t, lens, ints(new), ints(free), total, free_head=head, seq_lens=lens,
                                         free_head_out=head)
    assert t.tolist() == want[0] and lens.tolist() == want[1] and cu.tolist() == want[2]
    assert slots.tolist() == want[3] and head.tolist() == [want[4]]
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_assign_nothing(fd):
    t = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    lens, cu, slots, head = fd.fd_assign_pages(t, ints([5, 0]), ints([0, 0]), ints([]), 0)
    assert lens.tolist() == [5, 0] and cu.tolist() == [0, 0, 0] and slots.numel() == 0 and head.tolist() == [0]
    t = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    lens, cu, slots, head = fd.fd_assign_pages(t, ints([]), ints([]), ints([4]), 3, free_head=ints([1]))
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 3 and head.tolist() == [1]
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_assign_out_of_pages_and_bad_lengths(fd):
    t = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    lens, cu, slots, head = fd.fd_assign_pages(t, ints([0, 0, 0]), ints([64, 70, 1]), ints([9, 8]), 135)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_OUT_OF_PAGES
    assert t.tolist() == [[9, -1], [8, -1], [-1, -1]] and head.tolist() == [2]
    assert slots[:64].tolist() == list(range(9 * 64, 10 * 64))
    assert slots[64:128].tolist() == list(range(8 * 64, 9 * 64)) and slots[128:].tolist() == [-1] * 7
    # longer than the table, a negative length, and more tokens than slots
    t = torch.full((2, 2), -1, dtype=torch.int32, device="cuda")
    lens, cu, slots, head = fd.fd_assign_pages(t, ints([100, 0]), ints([40, 2]), ints([1, 2, 3]), 42)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_INVALID_ARG
    assert lens.tolist() == [128, 2] and cu.tolist() == [0, 40, 42]
    assert slots[28:40].tolist() == [-1] * 12 and slots[40:].tolist() == [64, 65]
    t = torch.full((2, 2), -1, dtype=torch.int32, device="cuda")
    fd.fd_assign_pages(t, ints([0, -3]), ints([-4, 5]), ints([1, 2, 3]), 5)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_INVALID_ARG
    slots = torch.full((8,), 77, dtype=torch.int64, device="cuda")
    fd.fd_assign_pages(t, ints([0, 0]), ints([3, 9]), ints([1, 2, 3]), 6, slots=slots[:6])
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_INVALID_ARG
    assert slots.tolist() == [64, 65, 66, 128, 129, 130, 77, 77]


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("T,Hkv,d", [(1, 1, 64), (1, 8, 128), (7, 3, 128), (300, 2, 64), (1000, 8, 128)])
@pytest.mark.parametrize("strided", [False, True])
def test_append(fd, T, Hkv, d, strided):
    g = generator(T)
    P = T // 64 + 4
    x = randn(g, T, 2 * Hkv * d + 40) if strided else randn(g, T, 2 * Hkv * d)
    k, v = x[:, :Hkv * d].unflatten(1, (Hkv, d)), x[:, Hkv * d:2 * Hkv * d].unflatten(1, (Hkv, d))
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    slots = torch.randperm(P * 64, generator=g, device="cuda")[:T]
    slots[::5] = -1
    kp, vp = randn(g, P, Hkv, 64, d), randn(g, P, Hkv, 64, d)
    want_k, want_v = kp.clone(), vp.clone()
    ok = slots >= 0
    want_k[slots[ok] // 64, :, slots[ok] % 64] = k[ok]
    want_v[slots[ok] // 64, :, slots[ok] % 64] = v[ok]
    fd.fd_append_kv_paged(k, v, slots, kp, vp)
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    # the fp8 cache gets the encoder's bytes
    codes = [torch.randint(0, 255, (P, Hkv, 64, d), generator=g, device="cuda").to(torch.uint8) for _ in range(2)]
    scales = [torch.rand((P, Hkv, 64), generator=g, device="cuda") for _ in range(2)]
    want = [c.clone() for c in codes], [s.clone() for s in scales]
    for i, y in enumerate((k, v)):
        c, s = fd.fd_quantize_kv_fp8(y.transpose(0, 1)[None].contiguous())  # [1, Hkv, T, d]
        want[0][i][slots[ok] // 64, :, slots[ok] % 64] = c[0].transpose(0, 1)[ok]
        want[1][i][slots[ok] // 64, :, slots[ok] % 64] = s[0].transpose(0, 1)[ok]
    fd.fd_append_kv_paged_fp8(k, v, slots, codes[0], scales[0], codes[1], scales[1])
    for i in range(2):
        assert torch.equal(codes[i], want[0][i]) and torch.equal(scales[i], want[1][i])
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_append_fp8_zero_and_extreme_rows(fd):
    k = torch.zeros((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    k[1] = 3e38
    k[2, 0, 5] = -1e-38
    k[3] = torch.linspace(-448, 448, 64).to(torch.bfloat16)
    codes = [torch.full((1, 1, 64, 64), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((1, 1, 64), 9.0, device="cuda") for _ in range(2)]
    fd.fd_append_kv_paged_fp8(k, k, ints([3, 2, 1, 0], torch.int64), codes[0], scales[0], codes[1], scales[1])
    c, s = fd.fd_quantize_kv_fp8(k.transpose(0, 1)[None].contiguous())
    assert torch.equal(codes[0][0, :, [3, 2, 1, 0]], c[0]) and torch.equal(scales[1][0, :, [3, 2, 1, 0]], s[0])
    assert torch.all(codes[0][0, 0, 4:] == 9)


def test_append_slot_outside_the_pool_is_reported(fd):
    g = generator(2)
    k, v = randn(g, 3, 2, 64), randn(g, 3, 2, 64)
    kp = torch.zeros((2, 2, 64, 64), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    fd.fd_append_kv_paged(k, v, ints([128, 5, 1 << 40], torch.int64), kp, vp)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_BAD_PAGE_TABLE
    assert torch.equal(kp[0, :, 5], k[1]) and int((kp != 0).any(-1).sum()) == 2
    assert fd.fd_device_status(clear=True) == fd.FD_OK


# ---------------------------------------------------------------- all together

@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (64, 6, 2)])
def test_serving_run(fd, d, Hq, Hkv):
    """A shared system prompt goes in once, then a batch of questions behind
    it, then decode steps captured in one graph; every output is checked
    against the 64-bit attention over the tokens as they were made."""
    g = generator(5)
    scale = 1 / math.sqrt(d)
    P, wide, B = 64, 24, 5
    kp = torch.full((P, Hkv, 64, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    free = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    head = ints([0])

    # the system prompt: 5 whole pages, attended from its packed keys
    n = 320
    q, sk, sv = randn(g, n, Hq, d), randn(g, n, Hkv, d), randn(g, n, Hkv, d)
    row = torch.full((1, wide), -1, dtype=torch.int32, device="cuda")
    _, cu, slots, _ = fd.fd_assign_pages(row, ints([0]), ints([n]), free, n, free_head=head, free_head_out=head)
    fd.fd_append_kv_paged(sk, sv, slots, kp, vp)
    out, lse = fd.fd_prefill_packed(q, sk, sv, cu)
    check_rows(out, lse, attend64(q, sk, sv, limits(n, n, True), scale))

    # the questions: their tables start with the shared pages
    table = row.repeat(B, 1)
    prefix = row[0, :5].clone()
    lens = ints([n] * B)
    asks = [1, 64, 100, 0, 129]
    T = sum(asks)
    q, k, v = randn(g, T, Hq, d), randn(g, T, Hkv, d), randn(g, T, Hkv, d)
    _, cu, slots, _ = fd.fd_assign_pages(table, lens, ints(asks), free, T, free_head=head, seq_lens=lens,
                                         free_head_out=head)
    fd.fd_append_kv_paged(k, v, slots, kp, vp)
    out, lse = fd.fd_prefill_paged(q, kp, vp, table, P, cu, lens)
    have = []
    for b, m in enumerate(asks):
        a = sum(asks[:b])
        have.append([torch.cat([sk, k[a:a + m]]), torch.cat([sv, v[a:a + m]])])
        check_rows(out[a:a + m], lse[a:a + m], attend64(q[a:a + m], *have[b], limits(m, n + m, True), scale))

    # decode steps: one graph, replayed
    q, k, v = randn(g, B, Hq, d), randn(g, B, Hkv, d), randn(g, B, Hkv, d)
    one = ints([1] * B)
    slots = torch.empty(B, dtype=torch.int64, device="cuda")
    cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    out = torch.empty((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, Hq), dtype=torch.float32, device="cuda")
    ws = torch.empty(fd.fd_shared_prefix_workspace_size(B, Hq, Hkv, n, (wide - 5) * 64, d), dtype=torch.uint8,
                     device="cuda")

    def step():
        fd.fd_assign_pages(table, lens, one, free, B, free_head=head, seq_lens=lens, cu_seqlens=cu, slots=slots,
                           free_head_out=head)
        fd.fd_append_kv_paged(k, v, slots, kp, vp)
        fd.fd_decode_paged_shared_prefix(q, kp, vp, prefix, table, P, lens, out=out, lse=lse, workspace=ws)

    def check():
        for b in range(B):
            for i, x in enumerate((k, v)):
                have[b][i] = torch.cat([have[b][i], x[b:b + 1]])
            check_rows(out[b:b + 1], lse[b:b + 1],
                       attend64(q[b:b + 1], *have[b], torch.tensor([have[b][0].shape[0]]), scale))

    step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(70):
        for x in (q, k, v):
            x.copy_(randn(g, *x.shape))
        graph.replay()
        torch.cuda.synchronize()
        check()
    assert fd.fd_device_status(clear=True) == fd.FD_OK
    want, wlse = fd.fd_decode_paged(q, kp, vp, table, P, lens)
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -6 and (lse - wlse).abs().max() < 1e-4
