"""Norms of rows whose squares pass binary32: differential results and rotated heads of any size that the
calls admit, beside ordinary rows, against the 64-bit formulas."""
import pytest
import torch

from diff_reference import check_diff, diff64, generator, ints, limits, rand, randn
from test_gpu_rope import check_bf16, table_of, turned

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("splits", [1, 3, 10])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (8, 1, 64), (4, 4, 128), (12, 2, 64)])
def test_decode(fd, Hq, Hkv, d, splits, dtype):
    """Values of 2^58 to 2^94 (their squares and the sums of d of them pass 2^128 from 2^60 on) and of 1."""
    g = generator(Hq + d)
    powers, L = [0, 58, 60, 61, 64, 80, 94], 700
    lens = [700, 1, 64, 300, 640, 65, 512]
    B = len(lens)
    q, k, v = randn(g, B, Hq, d), randn(g, B, Hkv, L, d), randn(g, B, Hkv, L, d)
    v *= 2.0 ** torch.tensor(powers, device="cuda", dtype=torch.float32)[:, None, None, None]
    lam, w = rand(g, 0.1, 0.5, Hq), rand(g, 0.2, 1.5, d)
    # (scores near 0: the maps share little more than their mean, whatever lam)
    out, lse = fd.fd_decode_dense_diff(q, k, v, lam, ints(lens), scale=0.01, norm_weight=w, num_splits=splits,
                                       out_dtype=dtype)
    plain, _ = fd.fd_decode_dense_diff(q, k, v, lam, ints(lens), scale=0.01, num_splits=splits, out_dtype="f32")
    for b, n in enumerate(lens):
        rows = slice(b, b + 1)
        args = (q[rows], k[b, :, :n].transpose(0, 1), v[b, :, :n].transpose(0, 1), lam, limits(1, n), 0.01)
        check_diff(out[rows], lse[rows], diff64(*args, w, rounding=2.0 ** -16), f"2^{powers[b]}")
        check_diff(plain[rows], None, diff64(*args, rounding=2.0 ** -16), f"2^{powers[b]} without norm")
    assert fd.fd_device_status(clear=True) == fd.FD_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("power", [58, 60, 61, 64, 78])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (7, 1, 64)])
def test_prompts(fd, Hq, Hkv, d, power, splits, dtype):
    """Ordinary rows and rows of large values in one tile: the values turn large behind the first 20 rows' keys."""
    g = generator(power + d)
    T, L = 70, 400
    q, k, v = randn(g, T, Hq, d), randn(g, L, Hkv, d), randn(g, L, Hkv, d)
    v[L - T + 20:] *= 2.0 ** power
    lam, w = rand(g, 0.1, 0.5, Hq), rand(g, 0.2, 1.5, d)
    cq, ck = ints([0, T]), ints([0, L])
    rounding = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -16
    out, lse = fd.fd_prefill_packed_diff(q, k, v, lam, cq, ck, scale=0.01, norm_weight=w, num_splits=splits,
                                         out_dtype=dtype)
    check_diff(out, lse, diff64(q, k, v, lam, limits(T, L), 0.01, w, rounding=rounding))
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_prompts_of_many_pieces(fd):
    """Large and ordinary values by KV head: a CTA's pieces follow each other in both orders."""
    g = generator(6)
    B, n, Hq, Hkv, d = 30, 150, 16, 8, 64
    T = B * n
    q, k, v = randn(g, T, Hq, d), randn(g, T, Hkv, d), randn(g, T, Hkv, d)
    v[:, ::3] *= 2.0 ** 70
    lam, w = rand(g, 0.1, 0.5, Hq), rand(g, 0.2, 1.5, d)
    out, lse = fd.fd_prefill_packed_diff(q, k, v, lam, ints([n * b for b in range(B + 1)]), scale=0.01, norm_weight=w,
                                         out_dtype="f32")
    for b in range(0, B, 7):
        a = slice(n * b, n * b + n)
        check_diff(out[a], lse[a], diff64(q[a], k[a], v[a], lam, limits(n, n), 0.01, w, rounding=2.0 ** -16))
    assert fd.fd_device_status(clear=True) == fd.FD_OK


SHAPES = [  # T, Hq, Hkv, d, rot, halves; the last ones with several rows a thread
    (6, 8, 2, 128, 64, False), (13, 3, 1, 64, 32, True), (9, 6, 3, 128, 64, True), (3000, 7, 3, 128, 128, False),
    (2501, 32, 8, 64, 32, True),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,halves", SHAPES)
def test_rotation_and_append(fd, T, Hq, Hkv, d, rot, halves, interleaved):
    """Heads of any finite size side by side, up to the largest bf16 values."""
    g = generator(T + d)
    n = d // 2 if halves else d
    H = Hq + Hkv
    x = randn(g, T, H * d // n, n, dtype=torch.float32).clamp(-1.9, 1.9)
    powers = torch.tensor([0, 59, 60, 62, 90, 127], device="cuda")
    x *= 2.0 ** powers[torch.randint(0, 6, x.shape[:2], generator=g, device="cuda")][..., None].double()
    x = x.to(torch.bfloat16).reshape(T, H, d)
    assert x.isfinite().all()
    q, k = x.split((Hq, Hkv), 1)
    v = randn(g, T, Hkv, d)
    table = table_of(rot, 300)
    pos = torch.randint(0, 300, (T,), generator=g, device="cuda", dtype=torch.int32)
    qw, kw = rand(g, 0.2, 1.5, n), rand(g, 0.2, 1.5, n)
    more = dict(positions=pos, q_weight=qw, k_weight=kw, norm_eps=1e-5, interleaved=interleaved, halves=halves)
    qr = turned(q, pos, table, qw, 1e-5, interleaved, halves)
    kr = turned(k, pos, table, kw, 1e-5, interleaved, halves)
    qo, ko = fd.fd_norm_rope(q, k, table, **more)
    check_bf16(qo, qr, "q")
    check_bf16(ko, kr, "k")
    P = T // 64 + 1
    slots = torch.randperm(P * 64, generator=g, device="cuda")[:T]
    page, row = slots // 64, slots % 64
    pools = [torch.zeros((P, Hkv, 64, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q2 = fd.fd_append_kv_paged_rope(q, k, v, slots, *pools, table, **more)[0]
    assert torch.equal(q2, qo) and torch.equal(pools[0][page, :, row], ko) and torch.equal(pools[1][page, :, row], v)
    codes = [torch.zeros((P, Hkv, 64, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((P, Hkv, 64), device="cuda") for _ in range(2)]
    q3 = fd.fd_append_kv_paged_rope_fp8(q, k, v, slots, codes[0], scales[0], codes[1], scales[1], table, **more)[0]
    assert torch.equal(q3, qo)
    z, E = kr
    s = scales[0][page, :, row].double()
    dec = codes[0].view(torch.float8_e4m3fn)[page, :, row].double() * s[..., None]
    allowed = E + (2.0 ** -4 + 2.0 ** -21) * (z.abs() + E) + 2.0 ** -10 * s[..., None] * (1 + 2.0 ** -20)
    assert ((dec - z).abs() <= allowed).all()
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_rows_that_are_not_finite_stay_alone(fd):
    g = generator(9)
    q = randn(g, 40, 8, 64)
    table, pos = table_of(64, 50), torch.arange(40, dtype=torch.int32, device="cuda")
    w = rand(g, 0.2, 1.5, 64)
    bad = q.clone()
    bad[3, 2, 5], bad[7, 0, 63] = float("nan"), float("inf")
    out, _ = fd.fd_norm_rope(bad, None, table, positions=pos, q_weight=w)
    want, _ = fd.fd_norm_rope(q, None, table, positions=pos, q_weight=w)
    rest = torch.ones((40, 8), dtype=torch.bool, device="cuda")
    rest[3, 2] = rest[7, 0] = False
    assert torch.equal(out[rest], want[rest])
    assert out[3, 2].isnan().all() and out[7, 0].isnan().any()
