"""Pools of a rotating append that lie side by side in one allocation, and pools that share memory with its rows."""
import pytest
import torch

from diff_reference import generator, ints, randn
from test_gpu_rope import table_of

pytestmark = pytest.mark.gpu


def test_side_by_side_is_fine_and_overlaps_are_refused(fd):
    g = generator(1)
    T, P, Hkv, d = 70, 3, 2, 64
    q, k, v = randn(g, T, 8, d).split((4, 2, 2), 1)
    table, pos = table_of(d, 100), torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.randperm(P * 64, generator=g, device="cuda")[:T]
    one, two = (torch.zeros((P, Hkv, 64, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    both = torch.zeros((2, P, Hkv, 64, d), dtype=torch.bfloat16, device="cuda")
    want = fd.fd_append_kv_paged_rope(q, k, v, slots, one, two, table, positions=pos)[0]
    got = fd.fd_append_kv_paged_rope(q, k, v, slots, both[0], both[1], table, positions=pos)[0]
    assert torch.equal(got, want) and torch.equal(both[0], one) and torch.equal(both[1], two)
    codes = torch.zeros((2, P, Hkv, 64, d), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, P, Hkv, 64), device="cuda")
    fd.fd_append_kv_paged_rope_fp8(None, k, v, slots, codes[0], scales[0], codes[1], scales[1], table, positions=pos)
    kept = both.clone()
    with pytest.raises(fd.FdError):
        fd.fd_append_kv_paged_rope(q, k, v, slots, both[0], both[0], table, positions=pos)
    rows = both[0].view(-1, Hkv, d)[:T]  # the keys to be stored are rows of the pool
    with pytest.raises(fd.FdError):
        fd.fd_append_kv_paged_rope(None, rows, v, slots, both[0], both[1], table, positions=pos)
    with pytest.raises(fd.FdError):
        fd.fd_append_kv_paged_rope_fp8(None, k, v, slots, codes[0], scales[0], codes[1], scales[0], table, positions=pos)
    assert torch.equal(both, kept)
    assert fd.fd_device_status(clear=True) == fd.FD_OK
