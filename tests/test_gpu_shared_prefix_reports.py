"""Lengths outside the table in a shared-prefix decode are clamped and
reported, whatever room the table leaves for own tokens."""
import pytest
import torch

from rows_reference import generator, randn, random_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("own", [0, 2])
@pytest.mark.parametrize("B,G", [(3, 2), (70, 4)])  # one tile of queries, and more
@pytest.mark.parametrize("bad", [1, 1 << 30, -1, -(1 << 31)])
def test_lengths_outside_the_table(fd, B, G, bad, own):
    g = generator(B)
    skip, Hkv, d = 3, 2, 64
    room = (skip + own) * 64
    kp, vp, table, pool = random_pool([room] * B, Hkv, d, g, skip=skip)
    q = randn(g, B, Hkv * G, d)
    prefix = table[0, :skip].clone()
    lens = torch.full((B,), room, dtype=torch.int32, device="cuda")
    want, wlse = fd.fd_decode_paged_shared_prefix(q, kp, vp, prefix, table, pool, lens)
    assert fd.fd_device_status(clear=True) == fd.FD_OK
    lens[B - 1] = bad if bad < 0 else room + min(bad, (1 << 31) - 1 - room)
    out, lse = fd.fd_decode_paged_shared_prefix(q, kp, vp, prefix, table, pool, lens)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_INVALID_ARG
    assert torch.equal(out[:-1], want[:-1]) and torch.equal(lse[:-1], wlse[:-1])
    if bad < 0:
        assert torch.all(out[-1] == 0) and torch.all(torch.isneginf(lse[-1]))
    else:
        assert torch.equal(out[-1], want[-1]) and torch.equal(lse[-1], wlse[-1])
    # the whole prefix and less of it are fine
    lens[:] = torch.arange(B, device="cuda") % (room + 1)
    fd.fd_decode_paged_shared_prefix(q, kp, vp, prefix, table, pool, lens)
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_dense_without_room_for_own_tokens(fd):
    g = generator(1)
    q, kp, vp = randn(g, 3, 4, 128), randn(g, 2, 200, 128), randn(g, 2, 200, 128)
    none = torch.empty((3, 2, 0, 128), dtype=torch.bfloat16, device="cuda")
    want, wlse = fd.fd_decode_dense_shared_prefix(q, kp, vp, none, none)
    for lens, status in (([0, 0, 0], fd.FD_OK), ([0, 5, 0], fd.FD_ERR_INVALID_ARG), ([-1, 0, 0], fd.FD_ERR_INVALID_ARG)):
        out, lse = fd.fd_decode_dense_shared_prefix(q, kp, vp, none, none,
                                                    torch.tensor(lens, dtype=torch.int32, device="cuda"))
        assert fd.fd_device_status(clear=True) == status
        assert torch.equal(out, want) and torch.equal(lse, wlse)
