"""Differential attention against the 64-bit formulas: single tokens over dense
and paged caches, packed prompts, tails over pages."""
import math

import pytest
import torch

from diff_reference import check_diff, diff64, generator, ints, limits, paged, rand, randn

pytestmark = pytest.mark.gpu
DEVICE_OK = 0


def weight_of(g, d, norm):
    return rand(g, 0.2, 1.5, d) if norm else None


def lam_of(g, T, Hq, per_token):
    return rand(g, 0.1, 0.6, T, Hq) if per_token else rand(g, 0.1, 0.6, Hq)


# decode: (Hq, Hkv, d, lengths, splits); groups of 1..8 query heads, chunks of one token to many tiles
DECODE = [
    (4, 4, 128, [1, 2, 63, 64, 65], 0),
    (4, 2, 128, [300, 0, 129, 1], 1),
    (6, 2, 64, [257, 1000, 0], 0),
    (8, 2, 128, [5000, 37, 640], 0),
    (5, 1, 128, [777, 64, 1], 3),
    (12, 2, 64, [1500, 3], 0),
    (7, 1, 64, [129, 4097], 7),
    (16, 2, 128, [2500, 2501, 0, 1], 0),
    (8, 1, 64, [64, 128, 192], 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,lens,splits", DECODE)
def test_decode(fd, Hq, Hkv, d, lens, splits, norm, dtype):
    g = generator(sum(lens) + Hq)
    B, L = len(lens), max(lens) + 5
    q = randn(g, B, Hq, d)
    kp, vp, table, P, have = paged(g, lens, Hkv, d)
    lam, w = lam_of(g, B, Hq, norm), weight_of(g, d, norm)
    scale = 1 / math.sqrt(d // 2)
    k = torch.full((B, Hkv, L, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    for b, n in enumerate(lens):
        k[b, :, :n], v[b, :, :n] = (x.transpose(0, 1) for x in have[b])
    got = {
        "paged": fd.fd_decode_paged_diff(q, kp, vp, lam, table, P, ints(lens), norm_weight=w, num_splits=splits,
                                         out_dtype=dtype),
        "dense": fd.fd_decode_dense_diff(q, k, v, lam, ints(lens), norm_weight=w, num_splits=splits, out_dtype=dtype),
    }
    for b, n in enumerate(lens):
        ref = diff64(q[b:b + 1], *have[b], lam[b:b + 1] if norm else lam, limits(1, n), scale, w,
                     rounding=2.0 ** -16)
        for name, (out, lse) in got.items():
            check_diff(out[b:b + 1], lse[b:b + 1], ref, f"{name} {b}")
            if n == 0:
                assert not out[b].any()
    assert fd.fd_device_status(clear=True) == DEVICE_OK


def test_decode_without_lengths_and_full_chunks(fd):
    g = generator(3)
    q, k, v, lam = randn(g, 2, 8, 128), randn(g, 2, 2, 640, 128), randn(g, 2, 2, 640, 128), rand(g, 0.1, 0.6, 8)
    out, lse = fd.fd_decode_dense_diff(q, k, v, lam, scale=0.2)
    one, none = fd.fd_decode_dense_diff(q, k, v, lam, scale=0.2, num_splits=1, want_lse=False)
    assert none is None
    for b in range(2):
        ref = diff64(q[b:b + 1], k[b].transpose(0, 1), v[b].transpose(0, 1), lam, limits(1, 640), 0.2,
                     rounding=2.0 ** -16)
        check_diff(out[b:b + 1], lse[b:b + 1], ref)
        check_diff(one[b:b + 1], None, ref)


def test_decode_lambda_zero_is_the_plain_decode_of_the_first_half(fd):
    """lam = 0 leaves the first map: fd_decode_dense with the second half of q cleared."""
    g = generator(4)
    q, k, v = randn(g, 3, 4, 128), randn(g, 3, 2, 700, 128), randn(g, 3, 2, 700, 128)
    first = q.clone()
    first[..., 64:] = 0
    lens = ints([700, 1, 333])
    want, wlse = fd.fd_decode_dense(first, k, v, lens, scale=0.125, out_dtype="f32")
    out, lse = fd.fd_decode_dense_diff(q, k, v, torch.zeros(4, device="cuda"), lens, scale=0.125, out_dtype="f32")
    # both round their weights to 2^-16 and their sums over 700 keys, |o| <= max |v| < 8
    assert (out - want).abs().max() <= 8 * 2 * (2.0 ** -16 + 700 * 2.0 ** -22)
    assert (lse[..., 0] - wlse).abs().max() <= 1e-4


# prompts: (Hq, Hkv, d, new tokens, cached tokens); groups that do and do not divide 128
PROMPTS = [
    (4, 4, 128, [1, 5, 60], [0, 0, 0]),
    (8, 2, 128, [130, 0, 257, 1], [0, 0, 0, 0]),
    (6, 2, 64, [33, 129, 64], [0, 0, 0]),
    (8, 2, 128, [7, 100, 1, 0], [300, 64, 1000, 77]),
    (10, 2, 64, [3, 129], [127, 1]),
    (8, 1, 128, [1, 1, 1], [5000, 0, 63]),
    (7, 1, 128, [40, 300], [12, 700]),
    (3, 3, 64, [513], [0]),
]


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("norm,dtype", [(False, "bf16"), (True, "bf16"), (True, "f32"), (False, "f32")])
@pytest.mark.parametrize("Hq,Hkv,d,new,ctx", PROMPTS)
def test_prompts(fd, Hq, Hkv, d, new, ctx, norm, dtype, splits):
    g = generator(sum(new) + Hq)
    lens = [n + c for n, c in zip(new, ctx)]
    kp, vp, table, P, have = paged(g, lens, Hkv, d)
    T = sum(new)
    q, lam, w = randn(g, T, Hq, d), lam_of(g, T, Hq, norm), weight_of(g, d, norm)
    cu = ints([sum(new[:b]) for b in range(len(new) + 1)])
    scale = 1 / math.sqrt(d // 2)
    got = {"paged": fd.fd_prefill_paged_diff(q, kp, vp, lam, table, P, cu, ints(lens), norm_weight=w,
                                             num_splits=splits, out_dtype=dtype)}
    k, v = (torch.cat([x[i] for x in have]) for i in (0, 1))
    ck = ints([sum(lens[:b]) for b in range(len(new) + 1)])
    got["packed"] = fd.fd_prefill_packed_diff(q, k, v, lam, cu, ck, norm_weight=w, num_splits=splits, out_dtype=dtype)
    rounding = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -16
    for b, n in enumerate(new):
        a = sum(new[:b])
        ref = diff64(q[a:a + n], *have[b], lam[a:a + n] if norm else lam, limits(n, lens[b]), scale, w,
                     rounding=rounding)
        for name, (out, lse) in got.items():
            check_diff(out[a:a + n], lse[a:a + n], ref, f"{name} {b}")
    assert fd.fd_device_status(clear=True) == DEVICE_OK


@pytest.mark.parametrize("lens", [[9] * 40, [(37 * b) % 2500 for b in range(40)]])
def test_drafts_of_many_sequences_in_parts_of_their_own_choice(fd, lens):
    Hq, Hkv, d, B = 16, 8, 64, len(lens)
    g = generator(32)
    kp, vp, table, P, have = paged(g, lens, Hkv, d, wide=400)  # room for many more keys than there are
    new = [min(4, n) for n in lens]
    T = sum(new)
    assert fd.fd_prefill_diff_num_splits(B, T, Hq, Hkv, table.shape[1] * 64, d) > 1
    q, lam, w = randn(g, T, Hq, d), lam_of(g, T, Hq, True), weight_of(g, d, True)
    cu = ints([sum(new[:b]) for b in range(B + 1)])
    out, lse = fd.fd_prefill_paged_diff(q, kp, vp, lam, table, P, cu, ints(lens), norm_weight=w)
    for b, n in enumerate(new):
        a = sum(new[:b])
        ref = diff64(q[a:a + n], *have[b], lam[a:a + n], limits(n, lens[b]), 1 / math.sqrt(32), w, rounding=2.0 ** -8)
        check_diff(out[a:a + n], lse[a:a + n], ref, str(b))
    assert fd.fd_device_status(clear=True) == DEVICE_OK


def test_prompts_without_the_causal_mask_and_rows_that_see_nothing(fd):
    g = generator(7)
    q, k, v, lam = randn(g, 70, 4, 64), randn(g, 50, 2, 64), randn(g, 50, 2, 64), rand(g, 0.1, 0.6, 4)
    w = rand(g, 0.2, 1.5, 64)
    cq, ck = ints([0, 30, 70]), ints([0, 50, 50])  # the second sequence has no keys
    out, lse = fd.fd_prefill_packed_diff(q, k, v, lam, cq, ck, causal=False, norm_weight=w)
    check_diff(out[:30], lse[:30], diff64(q[:30], k, v, lam, limits(30, 50, False), 1 / math.sqrt(32), w))
    assert not out[30:].any() and torch.isneginf(lse[30:]).all()
    # more queries than keys: the first 20 see none
    out, lse = fd.fd_prefill_packed_diff(q[:70], k, v, lam, ints([0, 70]), ints([0, 50]), norm_weight=w)
    assert not out[:20].any() and torch.isneginf(lse[:20]).all()
    check_diff(out[20:], lse[20:], diff64(q[20:], k, v, lam, limits(50, 50), 1 / math.sqrt(32), w))


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing_are_0_whatever_lambda_and_weights(fd, dtype, splits):
    Hq, Hkv, d, new, keys = 4, 2, 64, 40, 7
    g = generator(31)
    q, k, v = randn(g, new, Hq, d), randn(g, keys, Hkv, d), randn(g, keys, Hkv, d)
    bad = torch.full((new, Hq), float("nan"), device="cuda")
    w = torch.full((d,), float("inf"), device="cuda")
    out, lse = fd.fd_prefill_packed_diff(q, k, v, bad, ints([0, new]), ints([0, keys]), norm_weight=w, out_dtype=dtype,
                                         num_splits=splits)
    empty = new - keys
    assert (out[:empty] == 0).all() and (lse[:empty] == float("-inf")).all()
    assert out[empty:].isnan().all() and lse[empty:].isfinite().all()
    kc, vc = (x.transpose(0, 1)[None].repeat(2, 1, 1, 1).contiguous() for x in (k, v))
    out, lse = fd.fd_decode_dense_diff(q[:2], kc, vc, bad[:2], ints([0, keys]), norm_weight=w, out_dtype=dtype,
                                       num_splits=splits)
    assert (out[0] == 0).all() and (lse[0] == float("-inf")).all()
    assert out[1].isnan().all() and lse[1].isfinite().all()


def test_prompts_from_a_fused_projection_leave_other_rows_alone(fd):
    g = generator(8)
    Hq, Hkv, d, T = 6, 2, 128, 90
    qkv = randn(g, T, Hq + 2 * Hkv, d)
    q, k, v = qkv.split((Hq, Hkv, Hkv), dim=1)
    lam = rand(g, 0.1, 0.6, T, Hq + 3)[:, :Hq]  # strided too
    out = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq, 2), 7.0, device="cuda")
    for splits in (1, 2):
        fd.fd_prefill_packed_diff(q, k, v, lam, ints([10, 40, 80]), out=out, lse=lse, num_splits=splits)
        for a, b in ((10, 40), (40, 80)):
            check_diff(out[a:b], lse[a:b],
                       diff64(q[a:b], k[a:b], v[a:b], lam[a:b], limits(b - a, b - a), 1 / math.sqrt(d // 2)))
        for rows in (slice(0, 10), slice(80, T)):
            assert (out[rows] == 7).all() and (lse[rows] == 7).all()


@pytest.mark.parametrize("splits", [1, 4])
def test_bad_pages_are_left_out_and_reported(fd, splits):
    g = generator(9)
    kp, vp, table, P, have = paged(g, [400], 2, 128)
    table[0, 2], table[0, 4] = P, -5
    keep = torch.ones(400, dtype=torch.bool, device="cuda")
    keep[128:192] = keep[256:320] = False
    q, lam = randn(g, 1, 4, 128), rand(g, 0.1, 0.6, 4)
    ref = diff64(q, have[0][0][keep], have[0][1][keep], lam, limits(1, int(keep.sum())), 0.125)
    out, lse = fd.fd_decode_paged_diff(q, kp, vp, lam, table, P, ints([400]), num_splits=splits)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_BAD_PAGE_TABLE
    check_diff(out, lse, ref)
    out, lse = fd.fd_prefill_paged_diff(q, kp, vp, lam, table, P, ints([0, 1]), ints([400]), num_splits=splits)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_BAD_PAGE_TABLE
    check_diff(out, lse, ref)


def test_lengths_outside_the_table_are_clamped_and_reported(fd):
    g = generator(10)
    kp, vp, table, P, have = paged(g, [128, 128], 1, 64)
    q, lam = randn(g, 2, 2, 64), rand(g, 0.1, 0.6, 2)
    out, lse = fd.fd_decode_paged_diff(q, kp, vp, lam, table, P, ints([500, -3]))
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_INVALID_ARG
    check_diff(out[:1], lse[:1], diff64(q[:1], *have[0], lam, limits(1, 128), 1 / math.sqrt(32)))
    assert not out[1].any() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("half", [0, 1])
def test_a_score_that_is_not_finite_makes_its_rows_nan(fd, half, splits, bad):
    """In either map, and in no other head's row."""
    g = generator(11)
    kp, vp, table, P, have = paged(g, [300], 2, 128)
    q, lam, w = randn(g, 1, 4, 128).abs(), rand(g, 0.1, 0.6, 4), rand(g, 0.2, 1.5, 128)
    kp[table[0, 1], 0, 3, 64 * half] = bad  # token 67 of KV head 0
    for out, lse in (fd.fd_decode_paged_diff(q, kp, vp, lam, table, P, ints([300]), norm_weight=w, num_splits=splits),
                     fd.fd_prefill_paged_diff(q, kp, vp, lam, table, P, ints([0, 1]), ints([300]), norm_weight=w,
                                              num_splits=splits)):
        assert out[0, :2].isnan().all() and lse[0, :2, half].isnan().all()
        assert lse[0, :2, 1 - half].isfinite().all()
        check_diff(out[:, 2:], lse[:, 2:], diff64(q[:, 2:], have[0][0][:, 1:], have[0][1][:, 1:], lam[2:],
                                                  limits(1, 300), 0.125, w))


def test_scores_of_minus_infinity_weigh_nothing(fd):
    g = generator(12)
    k, v = randn(g, 1, 1, 200, 64), randn(g, 1, 1, 200, 64)
    q, lam = randn(g, 1, 2, 64).abs(), rand(g, 0.1, 0.6, 2)
    k[0, 0, 50:, 0] = -float("inf")   # map 0 sees the first 50 keys
    k[0, 0, :, 40] = -float("inf")    # map 1 none
    for splits in (1, 2):
        out, lse = fd.fd_decode_dense_diff(q, k, v, lam, num_splits=splits, out_dtype="f32")
        ref = diff64(q, k[0].transpose(0, 1)[:50].nan_to_num(neginf=0.0), v[0].transpose(0, 1)[:50],
                     torch.zeros_like(lam), limits(1, 50), 1 / math.sqrt(32), rounding=2.0 ** -16)
        assert torch.isneginf(lse[..., 1]).all()
        err = (out.double() - ref[0]).abs()
        assert (err <= ref[2] + 2.0 ** -24 * ref[0].abs()).all()
        out, z = fd.fd_prefill_packed_diff(q, k[0].transpose(0, 1).contiguous(), v[0].transpose(0, 1).contiguous(), lam,
                                           ints([0, 1]), ints([0, 200]), num_splits=splits, out_dtype="f32")
        assert torch.isneginf(z[..., 1]).all() and (z[..., 0] - lse[..., 0]).abs().max() <= 2 * ref[3].max()
        assert ((out.double() - ref[0]).abs() <= ref[2] + 2.0 ** -24 * ref[0].abs()).all()


def test_results_repeat_and_streams_do_not_disturb_each_other(fd):
    g = generator(13)
    lens = [3000, 1200, 5, 4000]
    kp, vp, table, P, _ = paged(g, lens, 2, 128)
    q, lam, w = randn(g, 4, 8, 128), rand(g, 0.1, 0.6, 8), rand(g, 0.2, 1.5, 128)
    qp, cu = randn(g, 400, 8, 128), ints([0, 100, 200, 205, 400])

    def both():
        return (fd.fd_decode_paged_diff(q, kp, vp, lam, table, P, ints(lens), norm_weight=w)
                + fd.fd_prefill_paged_diff(qp, kp, vp, lam, table, P, cu, ints(lens), norm_weight=w))

    want = both()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(both())
    torch.cuda.synchronize()
    for other in got:
        for x, y in zip(want, other):
            assert torch.equal(x, y)
    # an explicit stream
    out, lse = fd.fd_decode_paged_diff(q, kp, vp, lam, table, P, ints(lens), norm_weight=w, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_a_wait_that_runs_out_is_reported(fd):
    g = generator(14)
    k, v, q, lam = randn(g, 1, 2, 512, 128), randn(g, 1, 2, 512, 128), randn(g, 1, 4, 128), rand(g, 0.1, 0.6, 4)
    kt, vt = k[0].transpose(0, 1).contiguous(), v[0].transpose(0, 1).contiguous()
    calls = (lambda: fd.fd_decode_dense_diff(q, k, v, lam, num_splits=1),
             lambda: fd.fd_prefill_packed_diff(q, kt, vt, lam, ints([0, 1]), ints([0, 512]), num_splits=1))
    try:
        for call in calls:
            fd.fd_debug_inject_wait_timeout(2_000_000, 1)
            call()
            assert fd.fd_device_status(clear=True) == fd.FD_ERR_DEVICE_TIMEOUT
    finally:
        fd.fd_debug_inject_wait_timeout()
    ref = diff64(q, kt, vt, lam, limits(1, 512), 0.125)
    for call in calls:
        out, lse = call()
        check_diff(out, lse, ref)
    assert fd.fd_device_status(clear=True) == DEVICE_OK


def test_binding_refusals(fd):
    g = generator(15)
    q, k, v, lam = randn(g, 2, 4, 128), randn(g, 2, 2, 64, 128), randn(g, 2, 2, 64, 128), rand(g, 0, 1, 4)
    for bad in (lam[:3], lam.double(), lam.cpu(), rand(g, 0, 1, 3, 4), rand(g, 0, 1, 4, 2).T):
        with pytest.raises(ValueError):
            fd.fd_decode_dense_diff(q, k, v, bad)
    for kw in (dict(norm_weight=rand(g, 0, 1, 64)), dict(lse=torch.empty((2, 4), device="cuda")),
               dict(num_splits=2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            fd.fd_decode_dense_diff(q, k, v, lam, **kw)
    with pytest.raises(fd.FdError):
        fd.fd_decode_dense_diff(q, k, v, lam, norm_weight=rand(g, 0, 1, 128), norm_eps=0.0)
    with pytest.raises(fd.FdError):
        fd.fd_decode_dense_diff(q, k, v, lam, scale=-1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("case", ["rising", "jump", "first masked", "deep"])
def test_scores_far_above_the_first_ones(fd, case, splits, dtype):
    """Rows whose scores rise by hundreds behind their first keys, in one map or both, fall behind by hundreds, or
    start on a page that is left out."""
    g = generator(16)
    T, L, Hq, Hkv, d = 70, 700, 4, 2, 128
    kp, vp, table, P, have = paged(g, [L], Hkv, d)
    q, lam, w = randn(g, T, Hq, d), rand(g, 0.1, 0.6, Hq), rand(g, 0.2, 1.5, d)
    k, v = (x.clone() for x in have[0])
    q[..., 0] = q[..., 64] = 1.0
    up = torch.zeros(L, device="cuda")
    if case == "rising":
        up = torch.arange(L, device="cuda") * 2.0
    elif case == "jump":
        up[650:] = 3000.0
    elif case == "deep":
        up[100:] = -3000.0
    k[:, :, 0] = up.to(torch.bfloat16)[:, None]
    if case != "jump":
        k[:, :, 64] = up.to(torch.bfloat16)[:, None]
    keep = torch.ones(L, dtype=torch.bool, device="cuda")
    for j in range(-(-L // 64)):
        part = k[64 * j:64 * j + 64]
        kp[table[0, j], :, :part.shape[0]] = part.transpose(0, 1)
    bad = case == "first masked"
    if bad:
        table[0, 0] = -1
        keep[:64] = False
    lim = limits(T, L)
    out, lse = fd.fd_prefill_paged_diff(q, kp, vp, lam, table, P, ints([0, T]), ints([L]), norm_weight=w,
                                        num_splits=splits, out_dtype=dtype)
    assert fd.fd_device_status(clear=True) == (fd.FD_ERR_BAD_PAGE_TABLE if bad else fd.FD_OK)
    ref = diff64(q, k[keep], v[keep], lam, lim - 64 * bad, 0.125, w,
                 rounding=2.0 ** -8 if dtype == "bf16" else 2.0 ** -16)
    check_diff(out, lse, ref, case)
    one, z = fd.fd_decode_paged_diff(q[-1:].contiguous(), kp, vp, lam, table, P, ints([L]), norm_weight=w,
                                     num_splits=splits, out_dtype=dtype)
    fd.fd_device_status(clear=True)
    check_diff(one, z, diff64(q[-1:], k[keep], v[keep], lam, lim[-1:] - 64 * bad, 0.125, w, rounding=2.0 ** -16))


def test_many_pieces_once_more(fd):
    """Every piece of a CTA and the last one too."""
    g = generator(17)
    B, n, Hq, Hkv, d = 40, 300, 8, 8, 64
    T = B * n
    q, k, v, lam = randn(g, T, Hq, d), randn(g, T, Hkv, d), randn(g, T, Hkv, d), rand(g, 0.1, 0.6, Hq)
    q[..., 3] = 1.0
    rise = (torch.arange(T, device="cuda") % n).float()
    k[:, ::3, 3] = (rise * 4).to(torch.bfloat16)[:, None]  # some heads' pieces, not all
    cu = ints([n * b for b in range(B + 1)])
    out, lse = fd.fd_prefill_packed_diff(q, k, v, lam, cu)
    for b in range(0, B, 7):
        a = slice(n * b, n * b + n)
        check_diff(out[a], lse[a], diff64(q[a], k[a], v[a], lam, limits(n, n), 1 / math.sqrt(d // 2)))
    assert fd.fd_device_status(clear=True) == DEVICE_OK
