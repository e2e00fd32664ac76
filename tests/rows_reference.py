"""Plain 64-bit attention for the prompt and shared-prefix tests, with the
error bounds that the kernels' roundings allow.

For a row with weights w_j (softmax, sum 1) and W = sum_j w_j |v_j|:
  * a score is a binary32 sum of d products: off by at most
    es = d * 2^-23 * scale * max_j sum_c |q_c k_jc| (an ulp per addition, which
    also covers the rounding of scale * log2(e) * s)
  * 2^x and the rescaling factors: under 2^-20 relative per weight
  * the weights' rounding to bf16 before the product with V: 2^-8 relative
  * sums over n keys: n * 2^-23 relative (an ulp per addition)
  so |out - ref| <= (2^-8 + 2 es + 2^-20 + n 2^-22) W, then the output's own
  rounding (2^-8 relative for bf16, 2^-24 for float32), and
  |lse - ref| <= es + 2^-20 + n 2^-23 + 2^-22 |lse|.
"""
import torch


def attend64(q, k, v, limit, scale):
    """q [T, Hq, d], k, v [L, Hkv, d], limit [T] visible keys.  Returns
    (out [T, Hq, d], lse [T, Hq], out bound without the output rounding,
    lse bound), float64."""
    T, Hq, d = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    kk = k.double().repeat_interleave(G, dim=1)
    vv = v.double().repeat_interleave(G, dim=1)
    qq = q.double()
    hidden = torch.arange(L, device=q.device)[None, :] >= limit.to(q.device)[:, None]  # [T, L]
    # hidden keys take no part, whatever they hold
    seen = ~hidden.all(dim=0) if T else torch.zeros(L, dtype=torch.bool, device=q.device)
    kk = torch.where(seen[:, None, None], kk, 0.0)
    vv = torch.where(seen[:, None, None], vv, 0.0)
    s = torch.einsum("thd,lhd->htl", qq, kk) * scale
    a = torch.einsum("thd,lhd->htl", qq.abs(), kk.abs()) * scale
    s = s.masked_fill(hidden[None], float("-inf"))
    a = a.masked_fill(hidden[None], 0.0)
    lse = torch.logsumexp(s, dim=-1) if L else torch.full((Hq, T), float("-inf"), dtype=torch.float64, device=q.device)
    w = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    out = torch.einsum("htl,lhd->thd", w, vv)
    weight = torch.einsum("htl,lhd->thd", w, vv.abs())
    es = d * 2.0 ** -23 * (a.amax(dim=-1) if L else torch.zeros_like(lse))
    n = limit.to(q.device).double().clamp(min=0)[None, :]
    rel = 2.0 ** -8 + 2 * es + 2.0 ** -20 + n * 2.0 ** -22
    finite = torch.where(torch.isinf(lse), 0.0, lse)
    lse_bound = es + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * finite.abs()
    return out, lse.T, weight * rel.T[..., None], lse_bound.T


def check_rows(out, lse, ref, what=""):
    """`ref` as attend64 returns it."""
    want, want_lse, bound, lse_bound = ref
    half = torch.finfo(out.dtype).eps / 2
    got = out.double()
    assert torch.isfinite(got).all(), f"{what}: out is not finite"
    err = (got - want).abs()
    allowed = bound + half * (want.abs() + bound) + 1e-30
    assert (err <= allowed).all(), f"{what}: out off by {err.max().item()} (excess {(err - allowed).max().item()})"
    if lse is not None:
        empty = torch.isinf(want_lse)
        assert torch.equal(torch.isneginf(lse), empty), f"{what}: rows without keys differ"
        err = (lse.double() - want_lse).abs()[~empty]
        allowed = lse_bound[~empty]
        assert (err <= allowed).all(), f"{what}: lse off by {err.max().item() if err.numel() else 0}"


def limits(Lq, Lk, causal):
    n = torch.arange(Lq) + (Lk - Lq + 1) if causal else torch.full((Lq,), Lk)
    return n.clamp(0, max(Lk, 0))


def offsets(lens, device="cuda"):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=device)


def gather_pages(pages, row, L):
    """[L, Hkv, d] of one table row."""
    n = -(-L // 64)
    got = pages[row[:n].long()]
    return got.transpose(1, 2).reshape(-1, got.shape[1], got.shape[3])[:L]


def random_pool(lens, Hkv, d, g, skip=0, spare=3, poison=True):
    """Pools with every sequence's tokens in random pages, NaN wherever no
    token lies: (k_pages, v_pages, table [B, wide], pages).  The first `skip`
    pages of all rows are the same."""
    need = [max(0, -(-n // 64) - skip) for n in lens]
    wide = max(1, skip + max(need, default=0))
    total = skip + sum(need) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")
    table[:, :skip] = order[:skip]
    kp = torch.full((total, Hkv, 64, d), float("nan") if poison else 0.0, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()

    def fill(ids, rows):
        if rows:
            x = torch.randn((2, -(-rows // 64) * 64, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
            x[:, rows:] = float("nan") if poison else 0.0
            x = x.view(2, -1, 64, Hkv, d).transpose(2, 3)
            kp[ids.long()], vp[ids.long()] = x[0], x[1]

    fill(order[:skip], skip * 64)
    at = skip
    for b, n in enumerate(need):
        ids = order[at:at + n]
        table[b, skip:skip + n] = ids
        fill(ids, max(0, lens[b] - skip * 64))
        at += n
    return kp, vp, table, total


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g
