"""Norms and rotation of heads, and the same on the way into the paged cache,
against the 64-bit formulas.

With y the normalised head (relative error at most n 2^-25 + 2^-21: its sum of n
squares, rsqrtf, the products) a turned channel is y_a c - y_b s, off by at most
E = (|y_a c| + |y_b s|) (n 2^-25 + 2^-21 + 2^-22); then one rounding, half a step: bf16
2^-8 relative, e4m3 2^-4 relative or 2^-10 of the scale where that is more."""
import pytest
import torch

from diff_reference import generator, ints, rand, randn

pytestmark = pytest.mark.gpu


def table_of(rot, max_pos, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def turned(x, pos, table, weight, eps, interleaved, halves):
    """(values, error bound before the rounding) in 64 bits of x [T,H,d]."""
    T, H, d = x.shape
    y = x.double()
    if halves:
        y = y.reshape(T, 2 * H, d // 2)
    n = y.shape[-1]
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    rot = table.shape[1]
    c, s = (t[:, None, :] for t in table.double()[pos.long()].split(rot // 2, 1))
    out, size = y.clone(), y.abs()
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    size[..., a] = (y[..., a] * c).abs() + (y[..., b] * s).abs()
    size[..., b] = (y[..., b] * c).abs() + (y[..., a] * s).abs()
    rel = (n * 2.0 ** -25 + 2.0 ** -21 if weight is not None else 0.0) + 2.0 ** -22
    return out.reshape(T, H, d), size.reshape(T, H, d) * rel


def check_bf16(got, ref, what=""):
    want, bound = ref
    err = (got.double() - want).abs()
    allowed = bound + 2.0 ** -8 * (want.abs() + bound) + 1e-38
    assert (err <= allowed).all(), f"{what}: off by {err.max().item()} (excess {(err - allowed).max().item()})"


SHAPES = [  # T, Hq, Hkv, d, rot, halves
    (1, 4, 4, 128, 128, False),
    (5, 8, 2, 64, 64, False),
    (33, 6, 2, 128, 64, True),
    (130, 3, 1, 64, 32, True),
    (70, 32, 8, 128, 128, False),
    (257, 7, 7, 128, 32, False),
    (19, 64, 8, 128, 16, True),
    (8, 10, 5, 64, 16, False),
    # more rows than the GPU holds at once: several heads a thread
    (3000, 7, 3, 128, 128, False),
    (2501, 32, 8, 64, 32, True),
    (1777, 10, 5, 128, 64, True),
]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,halves", SHAPES)
def test_norm_rope(fd, T, Hq, Hkv, d, rot, halves, interleaved, norm):
    g = generator(T + d)
    qkv = randn(g, T, Hq + 2 * Hkv, d)
    q, k, _ = qkv.split((Hq, Hkv, Hkv), 1)
    n = d // 2 if halves else d
    table = table_of(rot, 700)
    pos = torch.randint(0, 700, (T,), generator=g, device="cuda", dtype=torch.int32)
    qw, kw = (rand(g, -1.5, 1.5, n), rand(g, -1.5, 1.5, n)) if norm else (None, None)
    more = dict(q_weight=qw, k_weight=kw, norm_eps=1e-5, interleaved=interleaved, halves=halves)
    qr = turned(q, pos, table, qw, 1e-5, interleaved, halves)
    kr = turned(k, pos, table, kw, 1e-5, interleaved, halves)
    qo, ko = fd.fd_norm_rope(q, k, table, positions=pos, **more)
    check_bf16(qo, qr, "q")
    check_bf16(ko, kr, "k")
    only, none = fd.fd_norm_rope(q, None, table, positions=pos, **more)
    assert none is None and torch.equal(only, qo)
    # in place, in the fused rows
    kept = qkv[:, Hq + Hkv:].clone()
    fd.fd_norm_rope(q, k, table, positions=pos, q_out=q, k_out=k, **more)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, Hq + Hkv:], kept)
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_tokens_left_out_and_positions_outside_the_table(fd):
    g = generator(1)
    q, k = randn(g, 6, 4, 64), randn(g, 6, 2, 64)
    table = table_of(64, 100)
    qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
    fd.fd_norm_rope(q, k, table, positions=ints([3, -1, 99, -100, 0, 5]), q_out=qo, k_out=ko)
    assert fd.fd_device_status(clear=True) == fd.FD_OK
    keep = [0, 2, 4, 5]
    check_bf16(qo[keep], turned(q[keep], ints([3, 99, 0, 5]), table, None, 0, False, False))
    assert (qo[[1, 3]] == 7).all() and (ko[[1, 3]] == 7).all()
    qo, _ = fd.fd_norm_rope(q, k, table, positions=ints([100, 1 << 30, 0, 0, 0, 99]))
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_INVALID_ARG
    check_bf16(qo, turned(q, ints([99, 99, 0, 0, 0, 99]), table, None, 0, False, False))


@pytest.mark.parametrize("B", [1, 3, 40, 1500])
def test_positions_from_offsets_and_lengths(fd, B):
    """Many short and empty sequences, and tokens in front of and behind all of them."""
    g = generator(B)
    new = torch.randint(0, 5, (B,), generator=g, device="cuda")
    new[B // 2] = 130
    ctx = torch.randint(0, 400, (B,), generator=g, device="cuda")
    cu = (torch.cat([ints([0], torch.int64), new.cumsum(0)]) + 3).to(torch.int32)
    T = int(cu[-1]) + 4
    q, k = randn(g, T, 3, 64), randn(g, T, 1, 64)
    table = table_of(64, 600)
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), new)
    pos = (ctx[seq] + torch.arange(T - 7, device="cuda") + 3 - cu[seq]).to(torch.int32)
    pos = torch.cat([ints([-1] * 3), pos, ints([-1] * 4)])
    outs = []
    for more in (dict(positions=pos), dict(cu_seqlens=cu, seq_lens=(ctx + new).to(torch.int32))):
        qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
        fd.fd_norm_rope(q, k, table, q_out=qo, k_out=ko, **more)
        outs.append((qo, ko))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    check_bf16(outs[1][0][3:-4], turned(q[3:-4], pos[3:-4], table, None, 0, False, False))
    assert (outs[1][0][:3] == 7).all() and (outs[1][1][-4:] == 7).all()
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_bad_offsets_and_lengths_are_reported(fd):
    g = generator(2)
    q, k = randn(g, 10, 2, 64), randn(g, 10, 2, 64)
    table = table_of(64, 50)
    for cu, lens in (([0, 5, 12], [5, 7]), ([0, 5, 10], [5, 3]), ([0, 5, 10], [5, 51])):
        qo, _ = fd.fd_norm_rope(q, k, table, cu_seqlens=ints(cu), seq_lens=ints(lens))
        assert fd.fd_device_status(clear=True) == fd.FD_ERR_INVALID_ARG, (cu, lens)
        check_bf16(qo[:5], turned(q[:5], ints([0, 1, 2, 3, 4]), table, None, 0, False, False))


def slots_of(g, T, P):
    s = torch.randperm(P * 64, generator=g, device="cuda")[:T]
    s[::7] = -1
    return s


@pytest.mark.parametrize("norm,interleaved", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,halves", SHAPES)
def test_append(fd, T, Hq, Hkv, d, rot, halves, interleaved, norm):
    g = generator(T + d + 1)
    q, k, v = randn(g, T, Hq + 2 * Hkv, d).split((Hq, Hkv, Hkv), 1)
    n = d // 2 if halves else d
    table = table_of(rot, 300)
    pos = torch.randint(0, 300, (T,), generator=g, device="cuda", dtype=torch.int32)
    qw, kw = (rand(g, -1.5, 1.5, n), rand(g, -1.5, 1.5, n)) if norm else (None, None)
    more = dict(positions=pos, q_weight=qw, k_weight=kw, norm_eps=1e-5, interleaved=interleaved, halves=halves)
    P = T // 64 + 2
    slots = slots_of(g, T, P)
    ok = slots >= 0
    page, row = slots[ok] // 64, slots[ok] % 64
    qo, ko = fd.fd_norm_rope(q, k, table, **more)
    # bf16: the same rows as the two calls one after the other
    want = [torch.full((P, Hkv, 64, d), 7, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    got = [x.clone() for x in want]
    fd.fd_append_kv_paged(ko, v, slots, *want)
    q2, kp, vp = fd.fd_append_kv_paged_rope(q, k, v, slots, *got, table, **more)
    assert torch.equal(q2, qo) and kp is got[0] and vp is got[1]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # e4m3: values as fd_append_kv_paged_fp8 stores them, keys from the unrounded rows
    codes = [torch.full((P, Hkv, 64, d), 9, dtype=torch.uint8, device="cuda") for _ in range(4)]
    scales = [torch.full((P, Hkv, 64), 9.0, device="cuda") for _ in range(4)]
    fd.fd_append_kv_paged_fp8(k, v, slots, codes[0], scales[0], codes[1], scales[1])
    q3 = fd.fd_append_kv_paged_rope_fp8(q, k, v, slots, codes[2], scales[2], codes[3], scales[3], table, **more)[0]
    assert torch.equal(q3, qo) and torch.equal(codes[3], codes[1]) and torch.equal(scales[3], scales[1])
    z, E = (x[ok] for x in turned(k, pos, table, kw, 1e-5, interleaved, halves))
    s = scales[2][page, :, row].double()
    top = z.abs().amax(-1)
    assert ((s - top / 448).abs() <= (E.amax(-1) + 2.0 ** -23 * top) / 448).all()
    dec = codes[2].view(torch.float8_e4m3fn)[page, :, row].double() * s[..., None]
    # (2^-21: the quotient's and the decoded product's own roundings)
    allowed = E + (2.0 ** -4 + 2.0 ** -21) * (z.abs() + E) + 2.0 ** -10 * s[..., None] * (1 + 2.0 ** -20)
    assert ((dec - z).abs() <= allowed).all()
    rest = torch.ones((P, 64), dtype=torch.bool, device="cuda")
    rest[page, row] = False
    assert (codes[2].transpose(1, 2)[rest] == 9).all() and (scales[2].transpose(1, 2)[rest] == 9).all()
    # the queries in place, in the fused rows
    kept = torch.cat([k, v], 1)
    fd.fd_append_kv_paged_rope(q, k, v, slots, *got, table, q_out=q, **more)
    assert torch.equal(q, qo) and torch.equal(torch.cat([k, v], 1), kept)
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_append_keys_and_values_alone_and_bad_slots(fd):
    g = generator(3)
    k, v = randn(g, 5, 2, 128), randn(g, 5, 2, 128)
    table = table_of(128, 10)
    pools = [torch.full((2, 2, 64, 128), 7, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = ints([0, 128, 127, -1, 5], torch.int64)
    none, _, _ = fd.fd_append_kv_paged_rope(None, k, v, slots, *pools, table, positions=ints([0, 1, 2, 3, -1]))
    assert none is None and fd.fd_device_status(clear=True) == fd.FD_ERR_BAD_PAGE_TABLE
    assert torch.equal(pools[0][0, :, 0], k[0])  # position 0 turns nothing
    check_bf16(pools[0][1, :, 63][None], turned(k[2:3], ints([2]), table, None, 0, False, False))
    assert torch.equal(pools[1][1, :, 63], v[2]) and torch.equal(pools[1][0, :, 0], v[0])
    for p in pools:  # nothing else: a slot outside, a negative one, a token left out
        assert int((p != 7).any(-1).sum()) == 4
    # a negative slot turns its query all the same
    q = randn(g, 5, 3, 128)
    qo, _, _ = fd.fd_append_kv_paged_rope(q, k, v, ints([-1] * 5, torch.int64), *pools, table,
                                          positions=ints([0, 1, 2, 3, 4]))
    check_bf16(qo, turned(q, ints([0, 1, 2, 3, 4]), table, None, 0, False, False))


def test_extreme_rows(fd):
    """Zero rows, the largest and the smallest values, values with NaN and infinities beside them."""
    k = torch.zeros((6, 1, 64), dtype=torch.bfloat16, device="cuda")
    k[1] = 3e38
    k[2, 0, 5] = -1e-38
    k[3, 0] = torch.linspace(-448, 448, 64)
    v = k.clone()
    v[4, 0, 7], v[5, 0, 8] = float("nan"), float("inf")
    table = table_of(64, 4)
    slots = torch.arange(6, device="cuda")
    codes = [torch.full((1, 1, 64, 64), 9, dtype=torch.uint8, device="cuda") for _ in range(4)]
    scales = [torch.full((1, 1, 64), 9.0, device="cuda") for _ in range(4)]
    fd.fd_append_kv_paged_fp8(k, v, slots, codes[0], scales[0], codes[1], scales[1])
    fd.fd_append_kv_paged_rope_fp8(None, k, v, slots, codes[2], scales[2], codes[3], scales[3], table,
                                   positions=torch.zeros(6, dtype=torch.int32, device="cuda"))
    for i in (0, 1):  # position 0: the same rows
        assert torch.equal(codes[i], codes[2 + i]) and torch.equal(scales[i], scales[2 + i])
    q, _ = fd.fd_norm_rope(k, None, table, positions=torch.zeros(6, dtype=torch.int32, device="cuda"))
    assert torch.equal(q, k)


def test_binding_refusals(fd):
    g = generator(4)
    q, k, v = randn(g, 5, 4, 64), randn(g, 5, 2, 64), randn(g, 5, 2, 64)
    table, pos = table_of(64, 10), ints([0, 1, 2, 3, 4])
    cu, lens = ints([0, 5]), ints([5])
    for kw in (dict(), dict(positions=pos, cu_seqlens=cu, seq_lens=lens), dict(cu_seqlens=cu), dict(positions=pos[:4]),
               dict(positions=pos.long()), dict(positions=pos, q_weight=rand(g, 0, 1, 32)),
               dict(positions=pos, halves=True, q_weight=rand(g, 0, 1, 64)),
               dict(positions=pos, q_out=q[:4])):
        with pytest.raises(ValueError):
            fd.fd_norm_rope(q, k, table, **kw)
    with pytest.raises(ValueError):
        fd.fd_norm_rope(q, None, table, positions=pos, k_out=k)
    with pytest.raises(fd.FdError):
        fd.fd_norm_rope(q, k, table, positions=pos, halves=True)  # rot beyond half a row
    with pytest.raises(fd.FdError):
        fd.fd_norm_rope(q, k, table[:, :24].contiguous(), positions=pos)
    long = randn(g, 10, 4, 64)
    with pytest.raises(fd.FdError):
        fd.fd_norm_rope(long[:5], k, table, positions=pos, q_out=long[1:6])
    with pytest.raises(fd.FdError):
        fd.fd_norm_rope(q, k, table, positions=pos, q_weight=rand(g, 0, 1, 64), norm_eps=0.0)
