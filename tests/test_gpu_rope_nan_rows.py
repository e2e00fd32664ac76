"""Key rows with NaN on their way into the e4m3 cache: the row stays NaN, and no other one changes."""
import pytest
import torch

from diff_reference import generator, rand, randn
from test_gpu_rope import table_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T", [40, 3000])
def test_nan_keys(fd, T, norm):
    g = generator(T)
    Hkv, d, P = 4, 64, T // 64 + 1
    k, v = randn(g, T, Hkv, d), randn(g, T, Hkv, d)
    table, pos = table_of(d, T), torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda")
    w = rand(g, 0.2, 1.5, d) if norm else None
    got = []
    bad = k.clone()
    bad[7, 1] = float("nan")
    bad[9, 2, 5] = float("nan")
    for x in (k, bad):
        codes = [torch.zeros((P, Hkv, 64, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros((P, Hkv, 64), device="cuda") for _ in range(2)]
        fd.fd_append_kv_paged_rope_fp8(None, x, v, slots, codes[0], scales[0], codes[1], scales[1], table, positions=pos,
                                       k_weight=w)
        rows = codes[0].view(torch.float8_e4m3fn).float() * scales[0][..., None]
        got.append(rows.transpose(1, 2).reshape(-1, Hkv, d)[:T])
    want, rows = got
    rest = torch.ones((T, Hkv), dtype=torch.bool, device="cuda")
    rest[7, 1] = rest[9, 2] = False
    assert torch.equal(rows[rest], want[rest])
    assert rows[7, 1].isnan().all()
    pair = [5, 5 + d // 2]  # the channel that is NaN, and the one that turns with it
    assert rows[9, 2].isnan().all() if norm else rows[9, 2][pair].isnan().all()
    if not norm:  # the others keep the scale of the largest that is a number
        others = [c for c in range(d) if c not in pair]
        assert rows[9, 2][others].isfinite().all()
    assert fd.fd_device_status(clear=True) == fd.FD_OK
