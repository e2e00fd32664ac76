"""Plain 64-bit differential attention for the tests, with the error bounds that
the kernels' roundings allow.

A map's output o_i and lse come from scores that are binary32 sums of n = d/2
products.  As in rows_reference: scores off by at most es = n 2^-23 scale
max_j sum_c |q_c k_jc|, 2^x and the rescaling under 2^-20 relative per weight,
the weights' rounding before the product with v `weight` relative (one bf16 term
2^-8, two 2^-16), sums over L keys L 2^-23 relative twice; so
  |o_i - ref| <= b_i = (weight + 2 es + 2^-20 + L 2^-22) sum_j w_j |v_j|.
The difference o = o_1 - lam o_2 rounds three times more:
  B = b_1 + |lam| b_2 + 2^-22 (|o_1| + |lam o_2|).
The norm y = w o / N, N = sqrt(mean(o^2) + eps): N moves by at most rms(B), so
with rho = rms(B) / N < 1
  |y' - y| <= |w| / (N (1 - rho)) (B + |o| rho) + (d 2^-25 + 2^-20) |y|
(its own sum of d squares, rsqrtf and three products).  Last the output's rounding,
half a step of its type.
"""
import torch


def maps64(q, k, v, limit, scale, weight):
    """One map: q, k [T or L, H, n], v [L, Hkv, d], limit [T] visible keys.
    Returns (out [T,Hq,d], lse [T,Hq], out bound, lse bound), float64."""
    T, Hq, n = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    limit = limit.to(q.device)
    hidden = torch.arange(L, device=q.device)[None, :] >= limit[:, None]
    seen = ~hidden.all(dim=0) if T else torch.zeros(L, dtype=torch.bool, device=q.device)
    kk = torch.where(seen[:, None, None], k.double(), 0.0).repeat_interleave(G, dim=1)
    vv = torch.where(seen[:, None, None], v.double(), 0.0).repeat_interleave(G, dim=1)
    s = torch.einsum("thc,lhc->htl", q.double(), kk) * scale
    a = torch.einsum("thc,lhc->htl", q.double().abs(), kk.abs()) * scale
    s = s.masked_fill(hidden[None], float("-inf"))
    a = a.masked_fill(hidden[None], 0.0)
    lse = torch.logsumexp(s, dim=-1) if L else torch.full((Hq, T), float("-inf"), dtype=torch.float64, device=q.device)
    w = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    out = torch.einsum("htl,lhd->thd", w, vv)
    heavy = torch.einsum("htl,lhd->thd", w, vv.abs())
    es = n * 2.0 ** -23 * (a.amax(dim=-1) if L else torch.zeros_like(lse))
    count = limit.double().clamp(min=0)[None, :]
    rel = weight + 2 * es + 2.0 ** -20 + count * 2.0 ** -22
    finite = torch.where(torch.isinf(lse), 0.0, lse)
    return out, lse.T, heavy * rel.T[..., None], (es + 2.0 ** -20 + count * 2.0 ** -23 + 2.0 ** -22 * finite.abs()).T


def diff64(q, k, v, lam, limit, scale, weight=None, eps=1e-5, rounding=2.0 ** -8):
    """q [T,Hq,d], k, v [L,Hkv,d], lam [Hq] or [T,Hq], weight [d] or None.
    Returns (out, lse [T,Hq,2], out bound without the output's rounding, lse bound)."""
    h = q.shape[-1] // 2
    o1, z1, b1, e1 = maps64(q[..., :h], k[..., :h], v, limit, scale, rounding)
    o2, z2, b2, e2 = maps64(q[..., h:], k[..., h:], v, limit, scale, rounding)
    lm = lam.double().expand(q.shape[:2])[..., None]
    o = o1 - lm * o2
    bound = b1 + lm.abs() * b2 + 2.0 ** -22 * (o1.abs() + (lm * o2).abs())
    if weight is not None:
        d = q.shape[-1]
        w = weight.double()
        N = torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
        rho = torch.sqrt((bound * bound).mean(-1, keepdim=True)) / N
        assert (rho < 0.5).all(), "these inputs say nothing about the norm"
        y = w * o / N
        bound = w.abs() / (N * (1 - rho)) * (bound + o.abs() * rho) + (d * 2.0 ** -25 + 2.0 ** -20) * y.abs()
        o = y
    return o, torch.stack([z1, z2], -1), bound, torch.stack([e1, e2], -1)


def check_diff(out, lse, ref, what=""):
    want, want_lse, bound, lse_bound = ref
    half = torch.finfo(out.dtype).eps / 2
    got = out.double()
    assert torch.isfinite(got).all(), f"{what}: out is not finite"
    err = (got - want).abs()
    allowed = bound + half * (want.abs() + bound) + 1e-30
    assert (err <= allowed).all(), f"{what}: out off by {err.max().item()} (excess {(err - allowed).max().item()})"
    if lse is not None:
        empty = torch.isinf(want_lse)
        assert torch.equal(torch.isneginf(lse), empty), f"{what}: maps without keys differ"
        off = (lse.double() - want_lse).abs()
        assert (off[~empty] <= lse_bound[~empty]).all(), f"{what}: lse off by {off[~empty].max().item()}"


def limits(n, L, causal=True):
    """Visible keys of the last n of L tokens."""
    if not causal:
        return torch.full((n,), L)
    return torch.arange(L - n + 1, L + 1).clamp(min=0)


# ---------------------------------------------------------------- inputs

def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def rand(g, lo, hi, *shape):
    return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def paged(g, lens, Hkv, d, spare=3, wide=0):
    """A pool whose pages hold the sequences in random order, NaN elsewhere:
    (k_pages, v_pages, table, num_pages, [(k, v) of each sequence [L,Hkv,d]])."""
    need = [-(-n // 64) for n in lens]
    P = sum(need) + spare
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need)) + wide), -1, dtype=torch.int32, device="cuda")
    kp = torch.full((P, Hkv, 64, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    have, at = [], 0
    for b, n in enumerate(lens):
        k, v = randn(g, n, Hkv, d), randn(g, n, Hkv, d)
        have.append((k, v))
        ids = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = ids
        for x, pool in ((k, kp), (v, vp)):
            for j, pg in enumerate(ids.tolist()):
                part = x[64 * j:64 * j + 64]
                pool[pg, :, :part.shape[0]] = part.transpose(0, 1)
    return kp, vp, table, P, have
