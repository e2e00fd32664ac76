"""Offsets of the rotating calls that run backwards or leave [0, T], wherever they stand."""
import pytest
import torch

from diff_reference import generator, ints, randn
from test_gpu_rope import check_bf16, table_of, turned

pytestmark = pytest.mark.gpu

T = 10
FAR = [0] + [3] * 3000
BAD = [
    [0, 8, 5, 10],             # the middle sequence, to which no token belongs
    [0, 50, 5, 10],
    [0, 5, 5, -1, 5, 10],
    [-2, 0, 5, 10],
    [0, 5, 12],
    FAR + [2, 3, 10],          # behind more empty sequences than the launch has threads
    FAR + [10, 11],
    [3, 3, 2, 10],
]


@pytest.mark.parametrize("cu", BAD, ids=lambda c: str(c if len(c) < 10 else c[-4:]))
def test_bad_offsets_are_reported(fd, cu):
    g = generator(len(cu))
    q, k, v = randn(g, T, 2, 64), randn(g, T, 2, 64), randn(g, T, 2, 64)
    table, lens = table_of(64, 50), ints([10] * (len(cu) - 1))
    fd.fd_norm_rope(q, k, table, cu_seqlens=ints(cu), seq_lens=lens)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_INVALID_ARG
    pools = [torch.zeros((1, 2, 64, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.arange(T, device="cuda")
    fd.fd_append_kv_paged_rope(None, k, v, slots, *pools, table, cu_seqlens=ints(cu), seq_lens=lens)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_INVALID_ARG


@pytest.mark.parametrize("cu", [[0, 10], [0, 0, 0, 4, 4, 10, 10], FAR + [10], [2, 2, 6]], ids=lambda c: str(c[-7:]))
def test_good_offsets_are_not(fd, cu):
    g = generator(len(cu))
    q, table = randn(g, T, 2, 64), table_of(64, 50)
    at = torch.tensor(cu, device="cuda")
    lens = (at[1:] - at[:-1] + 7).to(torch.int32)
    out = torch.full_like(q, 7)
    fd.fd_norm_rope(q, None, table, cu_seqlens=ints(cu), seq_lens=lens, q_out=out)
    assert fd.fd_device_status(clear=True) == fd.FD_OK
    pos = torch.cat([torch.arange(b - a, device="cuda") + 7 for a, b in zip(cu, cu[1:])])
    rows = slice(cu[0], cu[-1])
    check_bf16(out[rows], turned(q[rows], pos, table, None, 0, False, False))
    assert (out[:cu[0]] == 7).all() and (out[cu[-1]:] == 7).all()
