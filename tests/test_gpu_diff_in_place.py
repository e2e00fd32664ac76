"""Differential calls whose results would replace their queries: single tokens may,
prompts are refused."""
import pytest
import torch

from diff_reference import generator, ints, paged, rand, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("Hq", [4, 16])
def test_decode_in_place_of_its_queries(fd, Hq, splits):
    g = generator(Hq)
    lens = [300, 0, 1500]
    kp, vp, table, P, _ = paged(g, lens, 2, 128)
    q, lam, w = randn(g, 3, Hq, 128), rand(g, 0.1, 0.6, Hq), rand(g, 0.2, 1.5, 128)
    more = dict(norm_weight=w, num_splits=splits)
    want, lse = fd.fd_decode_paged_diff(q, kp, vp, lam, table, P, ints(lens), **more)
    out, z = fd.fd_decode_paged_diff(q, kp, vp, lam, table, P, ints(lens), out=q, **more)
    assert out is q and torch.equal(q, want) and torch.equal(z, lse)
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def test_prompts_refuse_it(fd):
    g = generator(5)
    kp, vp, table, P, have = paged(g, [100], 2, 64)
    q, lam = randn(g, 100, 4, 64), rand(g, 0.1, 0.6, 4)
    cu = ints([0, 100])
    kept = q.clone()
    with pytest.raises(fd.FdError):
        fd.fd_prefill_paged_diff(q, kp, vp, lam, table, P, cu, ints([100]), out=q)
    with pytest.raises(fd.FdError):
        fd.fd_prefill_packed_diff(q, *have[0], lam, cu, out=q)
    fused = randn(g, 100, 8, 64)  # rows whose first half the outputs would overwrite
    with pytest.raises(fd.FdError):
        fd.fd_prefill_packed_diff(fused[:, :4], *have[0], lam, cu, out=fused.view(200, 4, 64)[:100])
    assert torch.equal(q, kept)
