"""NaN and infinities: visible scores in the prompt attention and the
shared-prefix decode, rows of the fp8 append.

A NaN or +inf score makes its row NaN (softmax has no other answer), a score of
-inf weighs nothing, and every other row is what the 64-bit definition says,
however many parts the keys are cut into."""
import math

import pytest
import torch

from rows_reference import attend64, check_rows, gather_pages, generator, limits, offsets, randn, random_pool

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def expect_nan(got, ref, rows):
    """`rows` [T, Hq]: those are NaN in every channel, the others as in `ref`."""
    out, lse = got
    assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all()
    check_rows(out[~rows], lse[~rows], tuple(x[~rows] for x in ref))


def joined(refs):
    return tuple(torch.cat(x) for x in zip(*refs))


@pytest.mark.parametrize("num_splits", [0, 1, 2, 5])
@pytest.mark.parametrize("lens,d", [([300, 5, 200], 128), ([300, 5, 200], 64), ([20, 3], 128), ([20, 3], 64)], ids=str)
def test_packed_nan_key_and_query(fd, lens, d, num_splits):
    g = generator(1)
    T, Hq, Hkv = sum(lens), 8, 2
    q, k, v = randn(g, T, Hq, d), randn(g, T, Hkv, d), randn(g, T, Hkv, d)
    cu = offsets(lens)

    def call():
        return fd.fd_prefill_packed(q, k, v, cu, num_splits=num_splits)

    at = [sum(lens[:i]) for i in range(len(lens))]
    ref = joined([attend64(q[a:a + n], k[a:a + n], v[a:a + n], limits(n, n, True), 1 / math.sqrt(d))
                  for a, n in zip(at, lens)])
    # one channel of one key of the first sequence: its heads' queries from there on
    at = lens[0] * 2 // 3
    keep = k.clone()
    k[at, 1, 7] = NAN
    rows = torch.zeros((T, Hq), dtype=torch.bool, device="cuda")
    rows[at:lens[0], 4:] = True
    expect_nan(call(), ref, rows)
    # the very first key, alone in its row's view
    k.copy_(keep)
    k[0, 0] = NAN
    rows.zero_()
    rows[:lens[0], :4] = True
    expect_nan(call(), ref, rows)
    k.copy_(keep)
    # one channel of one query
    q[at, 3, d - 1] = NAN
    rows.zero_()
    rows[at, 3] = True
    expect_nan(call(), ref, rows)
    assert fd.fd_device_status(clear=True) == fd.FD_OK


@pytest.mark.parametrize("num_splits", [1, 3])
@pytest.mark.parametrize("T", [30, 400])
def test_packed_infinite_scores(fd, T, num_splits):
    g = generator(2)
    Hq, Hkv, d = 4, 2, 64
    q, k, v = randn(g, T, Hq, d), randn(g, T, Hkv, d), randn(g, T, Hkv, d)
    q[..., 5] = torch.where(q[..., 5] == 0, 1.0, q[..., 5].float()).to(q.dtype)
    at = T // 3
    gone = [x[torch.arange(T, device="cuda") != at] for x in (k, v)]
    k[at, :, 5] = INF
    out, lse = fd.fd_prefill_packed(q, k, v, offsets([T]), num_splits=num_splits)
    sees = (torch.arange(T, device="cuda") >= at)[:, None]
    up = sees & (q[..., 5] > 0)
    assert torch.isnan(out[up]).all() and torch.isnan(lse[up]).all()
    # elsewhere the key weighs nothing
    lim = limits(T, T, True) - (torch.arange(T) >= at).long()
    ref = attend64(q, *gone, lim, 1 / math.sqrt(d))
    rest = ~up
    check_rows(out[rest], lse[rest], tuple(x[rest] for x in ref))


@pytest.mark.parametrize("num_splits", [0, 1, 3])
@pytest.mark.parametrize("new,ctx", [([1, 1, 1], [700, 63, 3000]), ([200, 9], [500, 130])], ids=str)
def test_paged_nan_key(fd, new, ctx, num_splits):
    g = generator(3)
    total = [n + c for n, c in zip(new, ctx)]
    kp, vp, table, pool = random_pool(total, 2, 128, g)
    q = randn(g, sum(new), 8, 128)
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")

    def call():
        return fd.fd_prefill_paged(q, kp, vp, table, pool, offsets(new), lens, num_splits=num_splits)

    ref, a = [], 0
    for i, (n, L) in enumerate(zip(new, total)):
        ref.append(attend64(q[a:a + n], gather_pages(kp, table[i], L), gather_pages(vp, table[i], L),
                            limits(n, L, True), 1 / math.sqrt(128)))
        a += n
    ref = joined(ref)
    for pos in (0, 63, ctx[0] - 1):  # a cached key of the first sequence
        keep = kp.clone()
        kp[table[0, pos // 64].long(), 0, pos % 64, 3] = NAN
        rows = torch.zeros((sum(new), 8), dtype=torch.bool, device="cuda")
        rows[:new[0], :4] = True
        expect_nan(call(), ref, rows)
        kp.copy_(keep)


# G = 4 and 1; batches of one tile (own tokens in the same launch) and more (a launch of their own)
@pytest.mark.parametrize("num_splits", [0, 1, 3])
@pytest.mark.parametrize("B,Hq,d", [(5, 8, 128), (5, 2, 64), (70, 8, 128), (140, 2, 64), (140, 2, 128)])
def test_shared_prefix_nan_key(fd, B, Hq, d, num_splits):
    g = generator(B)
    skip, Hkv = 9, 2
    own = [[1, 200, 64, 0, 65][b % 5] for b in range(B)]
    lens = [skip * 64 + n for n in own]
    kp, vp, table, pool = random_pool(lens, Hkv, d, g, skip=skip)
    q = randn(g, B, Hq, d)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    prefix = table[0, :skip].clone()
    G = Hq // Hkv

    def call():
        return fd.fd_decode_paged_shared_prefix(q, kp, vp, prefix, table, pool, sl, num_splits=num_splits)

    ref = joined([attend64(q[b:b + 1], gather_pages(kp, table[b], n), gather_pages(vp, table[b], n), torch.tensor([n]),
                           1 / math.sqrt(d)) for b, n in enumerate(lens)])
    keep = kp.clone()
    for b, pos in ((0, 0), (1, 0), (1, 130), (4, 64)):  # an own key: that sequence's heads
        kp[table[b, skip + pos // 64].long(), 1, pos % 64, 3] = NAN
        rows = torch.zeros((B, Hq), dtype=torch.bool, device="cuda")
        rows[b, G:] = True
        expect_nan(call(), ref, rows)
        kp.copy_(keep)
    for pos in (0, 300):  # a shared key: everybody's
        kp[prefix[pos // 64].long(), 0, pos % 64, 0] = NAN
        rows = torch.zeros((B, Hq), dtype=torch.bool, device="cuda")
        rows[:, :G] = True
        expect_nan(call(), ref, rows)
        kp.copy_(keep)
    q[2, 1] = NAN
    rows = torch.zeros((B, Hq), dtype=torch.bool, device="cuda")
    rows[2, 1] = True  # sequence 2, its query alone
    expect_nan(call(), ref, rows)


@pytest.mark.parametrize("B", [5, 140])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_dense_shared_prefix_overflow(fd, B, bad):
    g = generator(7)
    Hkv, G, d, P, L = 2, 1, 64, 200, 100
    q = randn(g, B, Hkv * G, d)
    q[..., 9] = q[..., 9].abs() + 0.5
    kp, vp = randn(g, Hkv, P, d), randn(g, Hkv, P, d)
    k, v = randn(g, B, Hkv, L, d), randn(g, B, Hkv, L, d)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    lens[0] = 1
    ref = joined([attend64(q[b:b + 1], torch.cat([kp, k[b, :, :n]], 1).transpose(0, 1),
                           torch.cat([vp, v[b, :, :n]], 1).transpose(0, 1), torch.tensor([P + n]), 1 / math.sqrt(d))
                  for b, n in enumerate(lens.tolist())])
    k[0, 1, 0, 9] = bad  # the only own token of sequence 0
    rows = torch.zeros((B, Hkv * G), dtype=torch.bool, device="cuda")
    rows[0, 1] = True
    expect_nan(fd.fd_decode_dense_shared_prefix(q, kp, vp, k, v, lens), ref, rows)


@pytest.mark.parametrize("d", [64, 128])
def test_append_fp8_writes_the_encoders_bytes(fd, d):
    # the encoder's maximum skips NaN: a finite scale and one NaN code, nothing at all in a row of NaN;
    # an infinity makes the scale infinite
    g = generator(8)
    T, Hkv = 40, 3
    rows = randn(g, T, Hkv, d)
    neg = torch.tensor(-64, dtype=torch.int16, device="cuda").view(torch.bfloat16)  # 0xffc0
    assert torch.isnan(neg) and torch.signbit(neg)
    for t, (at, x) in enumerate(((5, NAN), (0, NAN), (d - 1, neg), (16, INF), (3, -INF), (slice(None), NAN),
                                 (slice(1, None), NAN), (slice(None), INF), (slice(0, 8), neg),
                                 (slice(None, None, 2), NAN))):
        rows[t, 1, at] = x
    rows[10], rows[10, :, 7] = 0.0, NAN
    rows[11, 0, 2], rows[11, 0, 9] = INF, NAN
    rows[12] *= 1e-38
    rows[12, 2, 4] = NAN
    rows[13] = 3e38
    rows[13, 0, 0], rows[13, 1, 40] = NAN, -INF
    slots = torch.randperm(64, generator=g, device="cuda")[:T]
    pools = [torch.full((1, Hkv, 64, d), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((1, Hkv, 64), 9.0, device="cuda") for _ in range(2)]
    fd.fd_append_kv_paged_fp8(rows, rows.flip(0), slots, pools[0], scales[0], pools[1], scales[1])
    for i, x in enumerate((rows, rows.flip(0))):
        codes, s = fd.fd_quantize_kv_fp8(x.transpose(0, 1)[None].contiguous())
        assert torch.equal(pools[i][0, :, slots], codes[0])
        assert torch.equal(scales[i][0, :, slots].view(torch.int32), s[0].view(torch.int32))
