"""Plans of the prompt and shared-prefix calls, as their workspace sizes show them."""
import pytest

import long_context_decode_split_gb300 as fd
from long_context_decode_split_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()


def records(B, Hq, Hkv, prefix_len, L_own, d, num_splits=0):
    """Partial results of a (sequence, query head)."""
    n = fd.fd_shared_prefix_workspace_size(B, Hq, Hkv, prefix_len, L_own, d, num_splits) - 256
    assert n > 0 and n % (B * Hq * (d + 2) * 4) == 0
    return n // (B * Hq * (d + 2) * 4)


@pytest.mark.parametrize("prefix_len", [64, 128])
@pytest.mark.parametrize("G", [1, 2])
def test_a_batch_as_large_as_the_prefix_is_nothing_special(prefix_len, G):
    # the own tokens go with the prefix while a tile holds the batch, whatever the prefix's length
    most = 128 // G
    for B in range(prefix_len - 1, prefix_len + 2):
        if B <= most:
            assert records(B, 2 * G, 2, prefix_len, 1 << 16, 64, 1) == records(B, 2 * G, 2, 1000, 1 << 16, 64, 1) == 17
        else:
            assert records(B, 2 * G, 2, prefix_len, 1 << 16, 64, 1) == records(B, 2 * G, 2, 1000, 1 << 16, 64, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,prefix_len", [(8, 32, 8, 8192), (32, 32, 8, 131072), (32, 32, 8, 32768),
                                                 (4, 8, 2, 2048), (16, 64, 8, 65536)])
def test_room_in_the_table_does_not_change_the_prefix_plan(B, Hq, Hkv, prefix_len):
    # beyond 4096 tokens a table's room says nothing about the lengths: the prefix keeps its parts
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def own_pieces(L):
        n = max(1, min(-(-L // 2048), 16, max(2, -(-8 * sms // (B * Hkv)))))
        chunk = -(-(-(-L // n)) // 128) * 128
        return -(-L // chunk)

    parts = [records(B, Hq, Hkv, prefix_len, room, 128) - own_pieces(room)
             for room in (4160, 8192, 1 << 15, 100032, 1 << 17, 1 << 20)]
    assert parts[0] > 1 and len(set(parts)) == 1, parts


@pytest.mark.gpu
@pytest.mark.parametrize("B,n,Hq,Hkv", [(6, 256, 4, 1), (4, 400, 4, 1), (3, 512, 2, 1), (10, 300, 1, 1)])
def test_packed_prompts_shorter_than_a_part_take_one(B, n, Hq, Hkv):
    # no sequence fills more than one part of 512 keys: the call needs no workspace
    import ctypes
    import torch
    x = torch.randn((B * n, Hq, 64), device="cuda").to(torch.bfloat16)
    k = x[:, :Hkv].contiguous()
    cu = torch.arange(B + 1, device="cuda", dtype=torch.int32) * n
    out = torch.empty_like(x)
    p = [ctypes.c_void_p(t.data_ptr()) for t in (x, k, cu, out)]
    st = fd.load().fd_prefill_packed(p[0], p[1], p[1], Hq * 64, Hkv * 64, Hkv * 64, p[2], p[2], B, B * n, B * n, Hq,
                                     Hkv, 64, 0.125, 1, 0, p[3], fd.FD_OUT_BF16, None, None, 0, None)
    torch.cuda.synchronize()
    assert st == fd.FD_OK
    want, _ = fd.fd_prefill_packed(x, k, k, cu, num_splits=1)
    assert torch.equal(out, want)
