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
@pytest.mark.parametrize("B,Hq,Hkv,prefix_len", [(8, 32, 8, 8192), (32, 32, 8, 131072), (32, 32, 8, 32768), (4, 8, 2, 2048),
                                                 (16, 64, 8, 65536)])
def test_room_in_the_table_does_not_change_the_prefix_plan(B, Hq, Hkv, prefix_len):
    # beyond 4096 tokens a table's room says nothing about the lengths: the prefix keeps its parts
    def own_pieces(L):
        blocks = -(-L // 128)
        n = 1 if blocks <= 16 else -(-blocks // 16) if blocks < 256 else 16
        chunk = -(-(-(-L // n)) // 128) * 128
        return -(-L // chunk)

    want = records(B, Hq, Hkv, prefix_len, 4096, 128) - own_pieces(4096)
    for room in (8192, 1 << 15, 100032, 1 << 17, 1 << 20):
        assert records(B, Hq, Hkv, prefix_len, room, 128) - own_pieces(room) == want, room
