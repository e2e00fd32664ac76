"""Prompt attention (packed and paged) against the 64-bit definition."""
import math

import pytest
import torch

from rows_reference import (attend64, check_rows, gather_pages, generator, limits, offsets, randn, random_pool)

pytestmark = pytest.mark.gpu


def run_packed(fd, lens_q, lens_k, Hq, Hkv, d, causal, seed, **kw):
    g = generator(seed)
    q, k, v = randn(g, sum(lens_q), Hq, d), randn(g, sum(lens_k), Hkv, d), randn(g, sum(lens_k), Hkv, d)
    cq, ck = offsets(lens_q), offsets(lens_k)
    out, lse = fd.fd_prefill_packed(q, k, v, cq, None if lens_q == lens_k else ck, causal=causal, **kw)
    a = b = 0
    for i, (n, m) in enumerate(zip(lens_q, lens_k)):
        ref = attend64(q[a:a + n], k[b:b + m], v[b:b + m], limits(n, m, causal), 1 / math.sqrt(d))
        check_rows(out[a:a + n], lse[a:a + n], ref, f"sequence {i} ({n} on {m})")
        a, b = a + n, b + m
    assert fd.fd_device_status(clear=True) == fd.FD_OK
    return out, lse


RAGGED = [1, 0, 63, 64, 65, 127, 128, 129, 300, 2, 257]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_packed_ragged(fd, G, d, causal):
    run_packed(fd, RAGGED, RAGGED, 2 * G, 2, d, causal, seed=G)


@pytest.mark.parametrize("lens", [[1], [2], [64], [1000], [2049], [0, 0, 5], [1] * 70, [31, 4000, 7]], ids=str)
def test_packed_lengths(fd, lens):
    run_packed(fd, lens, lens, 8, 2, 128, True, seed=3)


@pytest.mark.parametrize("num_splits", [1, 2, 5, 40])
def test_packed_splits(fd, num_splits):
    run_packed(fd, [3, 700, 64, 1], [3, 700, 64, 1], 6, 2, 128, True, seed=4, num_splits=num_splits)
    run_packed(fd, [5, 16], [3000, 900], 8, 1, 64, True, seed=5, num_splits=num_splits, out_dtype="f32")


@pytest.mark.parametrize("causal", [True, False])
def test_other_key_lengths_and_rows_without_keys(fd, causal):
    # more keys than queries, fewer (the first queries see nothing), none, and no queries
    out, lse = run_packed(fd, [10, 200, 130, 5, 0, 40], [300, 200, 60, 0, 77, 1], 8, 2, 128, causal, seed=6)
    if causal:
        assert torch.all(out[210:280] == 0) and torch.all(torch.isneginf(lse[210:280]))
    assert torch.all(out[340:345] == 0)


def test_float32_output_and_no_lse(fd):
    run_packed(fd, [200, 77], [200, 77], 4, 4, 64, True, seed=7, out_dtype="f32")
    g = generator(8)
    q, k, v = randn(g, 70, 8, 128), randn(g, 70, 8, 128), randn(g, 70, 8, 128)
    cu = offsets([70])
    out, lse = fd.fd_prefill_packed(q, k, v, cu, want_lse=False)
    assert lse is None
    assert torch.equal(out, fd.fd_prefill_packed(q, k, v, cu)[0])


def test_fused_projection_strides(fd):
    g = generator(9)
    lens, Hq, Hkv, d = [100, 33, 260], 8, 2, 128
    qkv = randn(g, sum(lens), (Hq + 2 * Hkv) * d + 24)  # a stride that is no multiple of a row
    q = qkv[:, :Hq * d].unflatten(1, (Hq, d))
    k = qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    v = qkv[:, (Hq + Hkv) * d:(Hq + 2 * Hkv) * d].unflatten(1, (Hkv, d))
    cu = offsets(lens)
    out, lse = fd.fd_prefill_packed(q, k, v, cu)
    want, wlse = fd.fd_prefill_packed(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_foreign_rows_do_not_leak(fd):
    # the neighbours' keys and values, and everything behind the last sequence, are NaN or infinite
    g = generator(10)
    lens, Hq, Hkv, d = [70, 190, 1, 65], 8, 2, 128
    T = sum(lens) + 300
    q, k, v = randn(g, T, Hq, d), randn(g, T, Hkv, d), randn(g, T, Hkv, d)
    cu = offsets(lens)
    a, b = 70, 260
    good = k[a:b].clone(), v[a:b].clone()
    k[:a], v[:a], k[b:], v[b:] = float("nan"), float("inf"), float("-inf"), float("nan")
    out = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, dtype=torch.float32, device="cuda")
    fd.fd_prefill_packed(q, k, v, cu, out=out, lse=lse)
    check_rows(out[a:b], lse[a:b], attend64(q[a:b], *good, limits(190, 190, True), 1 / math.sqrt(d)))
    assert torch.all(out[sum(lens):] == 7.0) and torch.all(lse[sum(lens):] == 7.0)


@pytest.mark.parametrize("num_splits", [2, 30])
def test_rows_of_no_sequence_are_left_alone_by_the_merge(fd, num_splits):
    g = generator(17)
    T, d = 900, 128
    q, k, v = randn(g, T, 4, d), randn(g, T, 2, d), randn(g, T, 2, d)
    cu = torch.tensor([100, 160, 700], dtype=torch.int32, device="cuda")
    n = fd.fd_prefill_workspace_size(2, T, 4, 2, T, d, num_splits)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN in every record
    out = torch.full((T, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 4), 7.0, dtype=torch.float32, device="cuda")
    fd.fd_prefill_packed(q, k, v, cu, num_splits=num_splits, out=out, lse=lse, workspace=ws)
    for a, b in ((100, 160), (160, 700)):
        check_rows(out[a:b], lse[a:b], attend64(q[a:b], k[a:b], v[a:b], limits(b - a, b - a, True), 1 / math.sqrt(d)))
    for a, b in ((0, 100), (700, 900)):
        assert torch.all(out[a:b] == 7.0) and torch.all(lse[a:b] == 7.0)


def test_scales_and_extreme_scores(fd):
    g = generator(11)
    for std, scale in ((30.0, 1.0), (1e-3, 0.1), (1.0, 1e-6)):
        q = (torch.randn((300, 4, 64), generator=g, device="cuda") * std).to(torch.bfloat16)
        k = (torch.randn((300, 2, 64), generator=g, device="cuda") * std).to(torch.bfloat16)
        v = randn(g, 300, 2, 64)
        out, lse = fd.fd_prefill_packed(q, k, v, offsets([300]), scale=scale)
        want, wlse, _, lb = attend64(q, k, v, limits(300, 300, True), scale)
        assert torch.isfinite(out).all()
        assert ((lse - wlse).abs() <= lb + 2.0 ** -22 * wlse.abs()).all()


def test_ascending_scores_rescale_every_block(fd):
    # every block of keys raises the maximum by far more than the block before
    g = generator(12)
    L, d = 1500, 128
    q = torch.zeros((L, 2, d), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    k = randn(g, L, 2, d)
    k[..., 0] = (torch.arange(L, device="cuda") // 16 * 8).to(torch.bfloat16)[:, None]
    v = randn(g, L, 2, d)
    out, lse = fd.fd_prefill_packed(q, k, v, offsets([L]), scale=0.5)
    check_rows(out, lse, attend64(q, k, v, limits(L, L, True), 0.5))
    # and descending: the first keys hold all the weight
    k[..., 0] = -k[..., 0]
    out, lse = fd.fd_prefill_packed(q, k, v, offsets([L]), scale=0.5)
    check_rows(out, lse, attend64(q, k, v, limits(L, L, True), 0.5))


def test_long_prompt_sampled(fd):
    g = generator(13)
    L, Hq, Hkv, d = 20000, 8, 2, 128
    q, k, v = randn(g, L, Hq, d), randn(g, L, Hkv, d), randn(g, L, Hkv, d)
    out, lse = fd.fd_prefill_packed(q, k, v, offsets([L]))
    for t in (0, 1, 127, 128, 4095, 9999, 16383, 19999):
        ref = attend64(q[t:t + 1], k[:t + 1], v[:t + 1], torch.tensor([t + 1]), 1 / math.sqrt(d))
        check_rows(out[t:t + 1], lse[t:t + 1], ref, f"token {t}")


def test_many_sequences(fd):
    g = torch.Generator().manual_seed(14)
    lens = torch.randint(0, 12, (2500,), generator=g).tolist()
    gg = generator(14)
    T, Hq, Hkv, d = sum(lens), 4, 2, 64
    q, k, v = randn(gg, T, Hq, d), randn(gg, T, Hkv, d), randn(gg, T, Hkv, d)
    cu = offsets(lens)
    out, lse = fd.fd_prefill_packed(q, k, v, cu)
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"))
    at = cu[seq].long()
    # every row attends at most 12 keys: gathered as [T, 12, ...]
    idx = at[:, None] + torch.arange(12, device="cuda")[None, :]
    ok = idx <= torch.arange(T, device="cuda")[:, None]
    kk, vv = (x.double()[idx.clamp(max=T - 1)].repeat_interleave(2, dim=2) for x in (k, v))
    s = torch.einsum("thd,tlhd->thl", q.double(), kk) / 8
    s = s.masked_fill(~ok[:, None, :], float("-inf"))
    w = torch.softmax(s, -1)
    want = torch.einsum("thl,tlhd->thd", w, vv)
    bound = torch.einsum("thl,tlhd->thd", w, vv.abs()) * (2.0 ** -8 + 1e-4)
    assert ((out.double() - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound)).all()
    assert ((lse - torch.logsumexp(s, -1)).abs() < 1e-4).all()


def test_offsets_out_of_range_are_reported(fd):
    g = generator(15)
    q, k, v = randn(g, 100, 4, 64), randn(g, 100, 4, 64), randn(g, 100, 4, 64)
    for bad in ([0, 50, 140], [-5, 50, 100], [0, 60, 40]):
        fd.fd_prefill_packed(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert fd.fd_device_status(clear=True) == fd.FD_ERR_INVALID_ARG
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_deterministic_and_captured(fd):
    g = generator(16)
    lens = [300, 5, 700]
    q, k, v = randn(g, sum(lens), 8, 128), randn(g, sum(lens), 2, 128), randn(g, sum(lens), 2, 128)
    cu = offsets(lens)
    want, wlse = fd.fd_prefill_packed(q, k, v, cu, num_splits=3)
    out, lse = torch.empty_like(want), torch.empty_like(wlse)
    n = fd.fd_prefill_workspace_size(len(lens), sum(lens), 8, 2, sum(lens), 128, 3)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fd.fd_prefill_packed(q, k, v, cu, num_splits=3, out=out, lse=lse, workspace=ws)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fd.fd_prefill_packed(q, k, v, cu, num_splits=3, out=out, lse=lse, workspace=ws)
    # new inputs and other lengths in the captured buffers
    q.copy_(randn(g, *q.shape))
    cu.copy_(offsets([4, 1000, 1]))
    want, wlse = fd.fd_prefill_packed(q, k, v, cu, num_splits=3)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_no_keys_at_all(fd):
    g = generator(18)
    q = randn(g, 37, 4, 64)
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = fd.fd_prefill_packed(q, k, k, offsets([30, 7]), offsets([0, 0]))
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    out, lse = fd.fd_prefill_packed(q[:0], k, k, offsets([]))
    assert out.shape == (0, 4, 64)
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_explicit_stream_and_wrong_tensors(fd):
    g = generator(19)
    q, k, v = randn(g, 300, 8, 128), randn(g, 300, 2, 128), randn(g, 300, 2, 128)
    cu = offsets([300])
    want, wlse = fd.fd_prefill_packed(q, k, v, cu, num_splits=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        # outputs and workspace are allocated on the stream that uses them: nothing is handed to
        # the current stream's work while this call still runs
        out, lse = fd.fd_prefill_packed(q, k, v, cu, num_splits=2, stream=side)
        torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    with pytest.raises(ValueError):
        fd.fd_prefill_packed(q, k.float(), v, cu)
    with pytest.raises(ValueError):
        fd.fd_prefill_packed(q, k, v.cpu(), cu)
    with pytest.raises(ValueError):
        fd.fd_prefill_packed(q, k, v[:299], cu)
    with pytest.raises(ValueError):
        fd.fd_prefill_packed(q, k[:, :, :64], v, cu)
    with pytest.raises(ValueError):
        fd.fd_prefill_packed(q.transpose(0, 1), k, v, cu)
    with pytest.raises(ValueError):
        fd.fd_prefill_packed(q, k[:1].expand(300, 2, 128), v, cu)
    with pytest.raises(ValueError):
        fd.fd_prefill_packed(q, k, v, cu.long())
    with pytest.raises(ValueError):
        fd.fd_prefill_packed(q, k, v, cu, num_splits=2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fd.FdError):
        fd.fd_prefill_packed(q, k, v, cu, scale=-1.0)


def test_two_calls_at_once(fd):
    # two streams, each call with its own results: nothing is shared between them
    g = generator(20)
    sets = [(randn(g, 3000, 8, 128), randn(g, 3000, 2, 128), randn(g, 3000, 2, 128)) for _ in range(2)]
    cu = offsets([1000, 2000])
    want = [fd.fd_prefill_packed(*s, cu) for s in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            got[i].append(fd.fd_prefill_packed(*sets[i], cu, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


# ---------------------------------------------------------------- paged

def run_paged(fd, new, ctx, Hq, Hkv, d, seed, causal=True, **kw):
    g = generator(seed)
    total = [n + c for n, c in zip(new, ctx)]
    kp, vp, table, pool = random_pool(total, Hkv, d, g)
    q = randn(g, sum(new), Hq, d)
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    out, lse = fd.fd_prefill_paged(q, kp, vp, table, pool, offsets(new), lens, causal=causal, **kw)
    a = 0
    for i, (n, L) in enumerate(zip(new, total)):
        k, v = gather_pages(kp, table[i], L), gather_pages(vp, table[i], L)
        check_rows(out[a:a + n], lse[a:a + n], attend64(q[a:a + n], k, v, limits(n, L, causal), 1 / math.sqrt(d)),
                   f"sequence {i} ({n} behind {L - n})")
        a += n
    assert fd.fd_device_status(clear=True) == fd.FD_OK
    return q, kp, vp, table, pool, lens, out, lse


@pytest.mark.parametrize("num_splits", [0, 1, 3])
@pytest.mark.parametrize("G,d", [(1, 64), (1, 128), (3, 128), (4, 64), (7, 128), (8, 128)])
def test_paged_tails(fd, G, d, num_splits):
    run_paged(fd, [1, 8, 64, 0, 130, 17, 300], [0, 63, 64, 100, 1, 2000, 129], 2 * G, 2, d, seed=G,
              num_splits=num_splits)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx,Hq,Hkv,d", [([64, 64], [20000, 100], 8, 2, 128), ([8, 8, 8, 8], [9000, 30, 0, 4000], 8, 2, 128),
                                              ([500], [6000], 16, 2, 64), ([1, 70, 0, 3], [5000, 1, 12000, 0], 7, 1, 128)])
def test_paged_parts_chosen_by_the_planner(fd, new, ctx, Hq, Hkv, d, causal):
    width = -(-max(n + c for n, c in zip(new, ctx)) // 64)
    assert fd.fd_prefill_num_splits(len(new), sum(new), Hq, Hkv, 64 * width, d) > 1
    run_paged(fd, new, ctx, Hq, Hkv, d, seed=sum(new), causal=causal)


def test_captured_parts_follow_the_lengths(fd):
    # the parts are cut on the device: a replay with other lengths is the call with those lengths
    g = generator(31)
    new, room = [40, 3, 80], [9000, 7000, 8000]
    kp, vp, table, pool = random_pool(room, 2, 128, g)
    q = randn(g, sum(new), 8, 128)
    cu = offsets(new)
    lens = torch.tensor(room, dtype=torch.int32, device="cuda")
    assert fd.fd_prefill_num_splits(3, sum(new), 8, 2, 64 * table.shape[1], 128) > 1
    out, lse = torch.empty_like(q), torch.empty(sum(new), 8, device="cuda")
    fd.fd_prefill_paged(q, kp, vp, table, pool, cu, lens, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fd.fd_prefill_paged(q, kp, vp, table, pool, cu, lens, out=out, lse=lse)
    for now in (room, [40, 6999, 300], [9000, 2, 0], [641, 3, 5000]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        want, wlse = fd.fd_prefill_paged(q, kp, vp, table, pool, cu, lens)
        assert torch.equal(out, want) and torch.equal(lse, wlse)
        a = 0
        for i, (n, L) in enumerate(zip(new, now)):
            k, v = gather_pages(kp, table[i], L), gather_pages(vp, table[i], L)
            check_rows(out[a:a + n], lse[a:a + n], attend64(q[a:a + n], k, v, limits(n, L, True), 128 ** -0.5))
            a += n
    assert fd.fd_device_status(clear=True) == fd.FD_OK


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("num_splits", [1, 2])
def test_keys_behind_the_causal_mask_may_hold_anything(fd, bad, num_splits):
    g = generator(32)
    q, k, v = randn(g, 333, 8, 128), randn(g, 333, 2, 128), randn(g, 333, 2, 128)
    cu = offsets([333])
    want, wlse = fd.fd_prefill_packed(q, k, v, cu, num_splits=num_splits)
    k[300:] = bad
    out, lse = fd.fd_prefill_packed(q, k, v, cu, num_splits=num_splits)
    assert torch.equal(out[:300], want[:300]) and torch.equal(lse[:300], wlse[:300])


def test_paged_not_causal_and_float32(fd):
    run_paged(fd, [5, 140], [300, 70], 8, 2, 128, seed=21, causal=False, out_dtype="f32")


def test_paged_single_token_is_the_decode(fd):
    q, kp, vp, table, pool, lens, out, lse = run_paged(fd, [1] * 6, [0, 62, 63, 64, 1000, 5000], 8, 2, 128, seed=22)
    want, wlse = fd.fd_decode_paged(q, kp, vp, table, pool, lens)
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -7 * 4
    assert (lse - wlse).abs().max() < 1e-4


def test_paged_empty_sequences_and_short_keys(fd):
    # seq_lens below the query count: the first queries see nothing
    g = generator(23)
    kp, vp, table, pool = random_pool([40, 100, 0], 2, 64, g)
    q = randn(g, 60 + 100 + 9, 4, 64)
    lens = torch.tensor([40, 100, 0], dtype=torch.int32, device="cuda")
    out, lse = fd.fd_prefill_paged(q, kp, vp, table, pool, offsets([60, 100, 9]), lens)
    a = 0
    for i, (n, L) in enumerate(zip([60, 100, 9], [40, 100, 0])):
        k, v = gather_pages(kp, table[i], L), gather_pages(vp, table[i], L)
        check_rows(out[a:a + n], lse[a:a + n], attend64(q[a:a + n], k, v, limits(n, L, True), 1 / 8))
        a += n
    assert torch.all(out[:20] == 0) and torch.all(out[160:] == 0)


@pytest.mark.parametrize("num_splits", [0, 2])
def test_paged_bad_page_is_skipped_and_reported(fd, num_splits):
    g = generator(24)
    new, total = [70, 10], [400, 333]
    kp, vp, table, pool = random_pool(total, 2, 128, g)
    q = randn(g, 80, 8, 128)
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    bad = table.clone()
    bad[0, 2], bad[1, 5] = pool + 9, -4
    out, lse = fd.fd_prefill_paged(q, kp, vp, bad, pool, offsets(new), lens, num_splits=num_splits)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_BAD_PAGE_TABLE
    a = 0
    for i, (n, L) in enumerate(zip(new, total)):
        k, v = gather_pages(kp, table[i], L), gather_pages(vp, table[i], L)
        gone = 2 if i == 0 else 5
        keep = torch.ones(L, dtype=torch.bool, device="cuda")
        keep[gone * 64:gone * 64 + 64] = False
        lim = limits(n, L, True)
        before = torch.cumsum(keep.long(), 0)
        lim = before[lim.to("cuda") - 1]
        check_rows(out[a:a + n], lse[a:a + n], attend64(q[a:a + n], k[keep], v[keep], lim, 1 / math.sqrt(128)))
        a += n
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_paged_lengths_outside_the_table_are_reported(fd):
    g = generator(25)
    kp, vp, table, pool = random_pool([128, 128], 2, 64, g)
    q = randn(g, 4, 4, 64)
    lens = torch.tensor([129, -1], dtype=torch.int32, device="cuda")
    out, _ = fd.fd_prefill_paged(q, kp, vp, table, pool, offsets([2, 2]), lens)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_INVALID_ARG
    assert torch.all(out[2:] == 0)
