"""A differential model's serving run: prompts and decode steps through pages,
rotation, append and attention, the decode steps captured in one graph."""
import math

import pytest
import torch

from diff_reference import check_diff, diff64, generator, ints, limits, rand, randn
from test_gpu_rope import check_bf16, table_of, turned

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (64, 5, 1)])
def test_serving_run(fd, d, Hq, Hkv):
    g = generator(5)
    B, P, wide, rot = 4, 60, 20, d // 2
    H = Hq + 2 * Hkv
    kp = torch.full((P, Hkv, 64, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    free = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    head, lens = ints([0]), ints([0] * B)
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    cs = table_of(rot, wide * 64)
    qw, kw, w = rand(g, 0.5, 1.5, d // 2), rand(g, 0.5, 1.5, d // 2), rand(g, 0.2, 1.5, d)
    lam = rand(g, 0.1, 0.6, Hq)
    scale = 1 / math.sqrt(d // 2)
    more = dict(q_weight=qw, k_weight=kw, norm_eps=1e-5, halves=True)

    def cached(b, n):
        ids = table[b, :-(-n // 64)].long()
        return (x[ids].transpose(1, 2).reshape(-1, Hkv, d)[:n] for x in (kp, vp))

    def check(qkv, cu, q, out, lse, new):
        """Rows turned, rows cached, attention over what is cached."""
        total = lens.tolist()
        for b, n in enumerate(new):
            a = int(cu[b])
            pos = torch.arange(total[b] - n, total[b], device="cuda")
            check_bf16(q[a:a + n], turned(qkv[a:a + n, :Hq], pos, cs, qw, 1e-5, False, True), "queries")
            k, v = cached(b, total[b])
            check_bf16(k[total[b] - n:], turned(qkv[a:a + n, Hq:Hq + Hkv], pos, cs, kw, 1e-5, False, True), "keys")
            assert torch.equal(v[total[b] - n:], qkv[a:a + n, Hq + Hkv:])
            check_diff(out[a:a + n], lse[a:a + n], diff64(q[a:a + n], k, v, lam, limits(n, total[b]), scale, w))

    new = [1, 130, 0, 64]
    T = sum(new) + 5  # a padded batch
    qkv = randn(g, T, H, d)
    _, cu, slots, _ = fd.fd_assign_pages(table, lens, ints(new), free, T, free_head=head, seq_lens=lens,
                                         free_head_out=head)
    q0 = torch.full((T, Hq, d), 7, dtype=torch.bfloat16, device="cuda")
    q, _, _ = fd.fd_append_kv_paged_rope(*qkv.split((Hq, Hkv, Hkv), 1), slots, kp, vp, cs, cu_seqlens=cu,
                                         seq_lens=lens, q_out=q0, **more)
    out = torch.full((T, Hq, d), 7, dtype=torch.bfloat16, device="cuda")
    _, lse = fd.fd_prefill_paged_diff(q, kp, vp, lam, table, P, cu, lens, norm_weight=w, out=out)
    check(qkv, cu, q, out, lse, new)
    assert (q[-5:] == 7).all() and (out[-5:] == 7).all()

    qkv = randn(g, B, H, d)
    one, slots = ints([1] * B), torch.empty(B, dtype=torch.int64, device="cuda")
    cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    q = torch.empty((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((B, Hq, 2), device="cuda")
    ws = torch.empty(fd.fd_decode_diff_workspace_size(B, Hq, Hkv, wide * 64, d, ragged=True), dtype=torch.uint8,
                     device="cuda")

    def step():
        fd.fd_assign_pages(table, lens, one, free, B, free_head=head, seq_lens=lens, cu_seqlens=cu, slots=slots,
                           free_head_out=head)
        fd.fd_append_kv_paged_rope(*qkv.split((Hq, Hkv, Hkv), 1), slots, kp, vp, cs, cu_seqlens=cu, seq_lens=lens,
                                   q_out=q, **more)
        fd.fd_decode_paged_diff(q, kp, vp, lam, table, P, lens, norm_weight=w, out=out, lse=lse, workspace=ws)

    step()
    check(qkv, cu, q, out, lse, [1] * B)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(70):
        qkv.copy_(randn(g, *qkv.shape))
        graph.replay()
        torch.cuda.synchronize()
        check(qkv, cu, q, out, lse, [1] * B)
    assert fd.fd_device_status(clear=True) == fd.FD_OK
