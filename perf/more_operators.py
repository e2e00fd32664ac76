"""Work cases of the differential attention and of the rotation on the way into
the cache: what they compute, in elementary torch operations, beside the calls
that a program makes of them.

Operators
  diff_decode   one new token per sequence against a paged or contiguous cache:
                the difference of two softmax maps, of the first halves of the
                query and key rows and of the second halves, over whole values
  diff_prompts  the same of many query tokens per sequence, packed (whole
                prompts) or behind cached tokens in 64-token pages
  norm_rope     norms of query and key heads (optional) and their rotation by
                position
  append_rope   the same with the keys, and the values beside them, written to
                their slots of a paged cache, in bf16 or as e4m3 codes with a
                scale per row

A case is a dict of plain values; lengths follow from its "lens_seed".
"""
import math
import random

import torch

own = False

PAGE = 64
BF16 = torch.bfloat16
EPS = 1e-5


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a few young conversations of a small model: launch latency is all there is
        dict(name="decode short", op="diff_decode", paged=True, B=4, lo=1, hi=300, Hq=8, Hkv=2, d=64, norm=False,
             per_token=False, lens_seed=1),
        # a serving engine's decode step over mixed contexts, results normalised
        dict(name="decode batch", op="diff_decode", paged=True, B=16, lo=4000, hi=32768, Hq=32, Hkv=8, d=128,
             norm=True, per_token=False, lens_seed=2),
        # one user's book-length context, contiguous
        dict(name="decode long", op="diff_decode", paged=False, B=1, lo=524288, hi=524288, Hq=32, Hkv=8, d=128,
             norm=True, per_token=False, lens_seed=3),
        # eight query heads to a KV head, weights of the second map from the token itself
        dict(name="decode wide groups", op="diff_decode", paged=True, B=8, lo=16000, hi=65536, Hq=64, Hkv=8, d=128,
             norm=False, per_token=True, lens_seed=4),
        # a handful of chat turns of a small model
        dict(name="prompts short", op="diff_prompts", paged=False, B=6, lo=5, hi=60, Hq=8, Hkv=2, d=64, norm=True,
             per_token=False, lens_seed=5),
        # a serving engine's prompt batch, ragged
        dict(name="prompts ragged", op="diff_prompts", paged=False, B=8, lo=257, hi=4095, Hq=32, Hkv=8, d=128,
             norm=True, per_token=False, lens_seed=6),
        # one document of 16K tokens
        dict(name="prompt 16K", op="diff_prompts", paged=False, B=1, lo=16384, hi=16384, Hq=32, Hkv=8, d=128,
             norm=False, per_token=False, lens_seed=7),
        # the next questions of running conversations, behind cached tokens
        dict(name="tails on context", op="diff_prompts", paged=True, B=8, lo=3, hi=700, ctx_lo=2000, ctx_hi=16000,
             Hq=32, Hkv=8, d=128, norm=True, per_token=True, lens_seed=8),
        # a drafted token each of three sequences, keys not cached yet; partial rotation of neighbouring pairs
        dict(name="rotate step", op="norm_rope", B=3, lo=1, hi=1, ctx_lo=10, ctx_hi=5000, Hq=8, Hkv=2, d=64, rot=32,
             norm=False, interleaved=True, halves=False, lens_seed=9),
        # queries and keys of a prompt batch, normalised per head
        dict(name="norm rotate prompts", op="norm_rope", B=8, lo=1000, hi=4000, ctx_lo=0, ctx_hi=0, Hq=32, Hkv=8,
             d=128, rot=128, norm=True, interleaved=False, halves=False, lens_seed=10),
        # the rows of a decode step of 256 sequences, for differential heads
        dict(name="append step", op="append_rope", fp8=False, B=256, lo=1, hi=1, ctx_lo=0, ctx_hi=32768, Hq=32, Hkv=8,
             d=128, rot=64, norm=False, interleaved=False, halves=True, lens_seed=11),
        # a batch of prompts into an e4m3 cache, with norms
        dict(name="append prompts fp8", op="append_rope", fp8=True, B=16, lo=1000, hi=3000, ctx_lo=0, ctx_hi=0, Hq=32,
             Hkv=8, d=128, rot=128, norm=True, interleaved=False, halves=False, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("diff_decode", "diff_prompts", "norm_rope", "append_rope"))
    seed = rng.randrange(1 << 30)
    Hq, Hkv = rng.choice(((4, 4), (8, 2), (12, 4), (16, 4), (10, 2), (32, 8), (28, 4), (64, 8)))
    d = rng.choice((64, 128, 128))
    heads = dict(Hq=Hq, Hkv=Hkv, d=d, lens_seed=seed)
    if op == "diff_decode":
        B = _log(rng, 1, 32)
        hi = _log(rng, 1, 400000 // B)
        return dict(op=op, paged=rng.random() < 0.7, B=B, lo=_log(rng, 1, hi), hi=hi, norm=rng.random() < 0.5,
                    per_token=rng.random() < 0.3, **heads)
    if op == "diff_prompts":
        paged = rng.random() < 0.5
        B = _log(rng, 1, 16)
        hi = _log(rng, 1, 700 if paged else 8000 // max(1, B // 2))
        ctx = _log(rng, 1, 40000 // B) if paged else 0
        return dict(op=op, paged=paged, B=B, lo=_log(rng, 1, hi), hi=hi, ctx_lo=ctx // 4, ctx_hi=ctx,
                    norm=rng.random() < 0.5, per_token=rng.random() < 0.3, **heads)
    B = _log(rng, 1, 300)
    hi = _log(rng, 1, max(1, 30000 // B))
    ctx = _log(rng, 1, 30000)
    halves = rng.random() < 0.4
    dh = d // 2 if halves else d
    more = dict(B=B, lo=_log(rng, 1, hi), hi=hi, ctx_lo=0, ctx_hi=ctx, rot=rng.choice((dh, dh, dh // 2)),
                norm=rng.random() < 0.5, interleaved=rng.random() < 0.3, halves=halves, **heads)
    if op == "append_rope":
        more["fp8"] = rng.random() < 0.5
    return dict(op=op, **more)


def _lens(case):
    """(new tokens, earlier tokens) of every sequence; the last one has the
    case's full length."""
    rng = random.Random(case["lens_seed"])
    new = [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    ctx = [rng.randint(case.get("ctx_lo", 0), case.get("ctx_hi", 0)) for _ in range(case["B"])]
    new[-1] = case["hi"]
    return new, ctx


def work(case):
    new, ctx = _lens(case)
    op, Hq, Hkv, d = case["op"], case["Hq"], case["Hkv"], case["d"]
    if op == "diff_decode":
        # q and out, both lse, the cache
        return {"bytes": 4 * d * Hkv * sum(new) + case["B"] * Hq * (4 * d + 8), "flops": 6 * d * Hq * sum(new)}
    if op == "diff_prompts":
        pairs = sum(n * (n + 1) // 2 + n * c for n, c in zip(new, ctx))
        return {"bytes": 4 * d * Hkv * (sum(new) + sum(ctx)) + sum(new) * Hq * (4 * d + 8), "flops": 6 * d * Hq * pairs}
    T = sum(new)
    at = set()
    for n, c in zip(new, ctx):
        at.update(range(c, c + n))
    bytes_ = T * Hq * 4 * d + 4 * case["rot"] * len(at)
    if op == "norm_rope":
        return {"bytes": bytes_ + T * (Hkv * 4 * d + 4), "flops": 0}
    return {"bytes": bytes_ + 2 * T * Hkv * (2 * d + (d + 4 if case["fp8"] else 2 * d)) + 8 * T, "flops": 0}


# ---------------------------------------------------------------- the inputs

def _rows(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(BF16)


def _keys(g, *shape):
    """Keys whose first channels carry a common offset, as those of trained
    models do: scores share a large part and spread by a few units."""
    k = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    k[..., :4] += 2.0
    return k.to(BF16)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _tables(g, lens, spare=2):
    """Pages of a pool in random order: (table [B, max_pages], pages in the pool)."""
    need = [-(-n // PAGE) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _uniform(g, lo, hi, *shape):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32) * (hi - lo) + lo


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    new, ctx = _lens(case)
    op, B, Hq, Hkv, d = (case[n] for n in ("op", "B", "Hq", "Hkv", "d"))
    s = dict(case)
    total = [n + c for n, c in zip(new, ctx)]
    if op in ("diff_decode", "diff_prompts"):
        T = B if op == "diff_decode" else sum(new)
        s["scale"] = 1.0 / math.sqrt(d // 2)
        s["new"], s["ctx"], s["most"] = new, ctx, max(total)
        s["q"] = _rows(g, T, Hq, d)
        s["lam"] = _uniform(g, 0.2, 0.8, T, Hq) if case["per_token"] else _uniform(g, 0.2, 0.8, Hq)
        s["weight"] = _uniform(g, 0.1, 0.6, d) if case["norm"] else None
        s["lens"], s["cu"] = _ints(total), _ints(_offsets(new))
        if case["paged"]:
            s["table"], s["pool"] = _tables(g, total)
            s["k"], s["v"] = _keys(g, s["pool"], Hkv, PAGE, d), _rows(g, s["pool"], Hkv, PAGE, d)
        elif op == "diff_decode":
            s["k"], s["v"] = _keys(g, B, Hkv, s["most"], d), _rows(g, B, Hkv, s["most"], d)
        else:
            s["k"], s["v"] = _keys(g, T, Hkv, d), _rows(g, T, Hkv, d)
        return s
    T, rot, dh = sum(new), case["rot"], d // 2 if case["halves"] else d
    # a fused projection's rows, and what a model keeps: tables of its rotation, weights of its norms
    s["qkv"] = _rows(g, T, Hq + 2 * Hkv, d)
    freq = 500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(max(total), device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()
    for n in ("q_weight", "k_weight"):
        s[n] = _uniform(g, 0.5, 1.5, dh) if case["norm"] else None
    pos = torch.cat([torch.arange(c, c + n, device="cuda") for n, c in zip(new, ctx)])
    s["positions"] = pos.to(torch.int32)
    s["cu"], s["lens"] = _ints(_offsets(new)), _ints(total)
    if op == "append_rope":
        # pages that hold the new tokens only: where the earlier ones lie does not matter here
        first = [c // PAGE for c in ctx]
        table, pool = _tables(g, [t - f * PAGE for t, f in zip(total, first)])
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), _ints(new, torch.int64))
        page = table[seq, pos // PAGE - _ints(first, torch.int64)[seq]]
        s["slots"] = page.to(torch.int64) * PAGE + pos % PAGE
        for n in "kv":
            s[n + "_pages"] = torch.zeros((pool, Hkv, PAGE, d), dtype=torch.uint8 if case["fp8"] else BF16,
                                          device="cuda")
            s[n + "_scales"] = torch.zeros((pool, Hkv, PAGE), dtype=torch.float32, device="cuda")
    return s


def _split(s):
    return s["qkv"].split((s["Hq"], s["Hkv"], s["Hkv"]), dim=1)


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import long_context_decode_split_gb300 as fd
    op = s["op"]
    if op in ("diff_decode", "diff_prompts"):
        more = dict(scale=s["scale"], norm_weight=s["weight"], norm_eps=EPS)
        if op == "diff_decode":
            if s["paged"]:
                return fd.fd_decode_paged_diff(s["q"], s["k"], s["v"], s["lam"], s["table"], s["pool"], s["lens"],
                                               **more)
            return fd.fd_decode_dense_diff(s["q"], s["k"], s["v"], s["lam"], s["lens"], **more)
        if s["paged"]:
            return fd.fd_prefill_paged_diff(s["q"], s["k"], s["v"], s["lam"], s["table"], s["pool"], s["cu"],
                                            s["lens"], **more)
        return fd.fd_prefill_packed_diff(s["q"], s["k"], s["v"], s["lam"], s["cu"], **more)
    q, k, v = _split(s)
    more = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], norm_eps=EPS, interleaved=s["interleaved"],
                halves=s["halves"])
    if op == "norm_rope":
        return fd.fd_norm_rope(q, k, s["cos_sin"], positions=s["positions"], **more)
    more.update(cu_seqlens=s["cu"], seq_lens=s["lens"])
    if s["fp8"]:
        q = fd.fd_append_kv_paged_rope_fp8(q, k, v, s["slots"], s["k_pages"], s["k_scales"], s["v_pages"],
                                           s["v_scales"], s["cos_sin"], **more)[0]
    else:
        q = fd.fd_append_kv_paged_rope(q, k, v, s["slots"], s["k_pages"], s["v_pages"], s["cos_sin"], **more)[0]
    return (q,) + _pools(s)


def _pools(s):
    if s["fp8"]:
        e4m3 = torch.float8_e4m3fn
        return s["k_pages"].view(e4m3), s["k_scales"], s["v_pages"].view(e4m3), s["v_scales"]
    return s["k_pages"], s["v_pages"]


def _plain(s):
    op = s["op"]
    if op == "diff_decode":
        return _plain_decode(s)
    if op == "diff_prompts":
        return _plain_prompts(s)
    q, k, v = _split(s)
    pos = s["positions"].long()
    q, k = _plain_rope(s, q, pos, s["q_weight"]), _plain_rope(s, k, pos, s["k_weight"])
    if op == "norm_rope":
        return q.to(BF16), k.to(BF16)
    page, row = s["slots"] // PAGE, s["slots"] % PAGE
    for n, x in (("k", k), ("v", v)):
        if s["fp8"]:
            x = x.float()
            scale = x.abs().amax(dim=-1) / 448
            x = torch.where(scale[..., None] > 0, x / scale[..., None], 0.0).to(torch.float8_e4m3fn).view(torch.uint8)
            s[n + "_scales"][page, :, row] = scale
        s[n + "_pages"][page, :, row] = x.to(s[n + "_pages"].dtype)
    return (q.to(BF16),) + _pools(s)


def _plain_rope(s, x, pos, weight):
    """Norm and rotation of the heads x [T, H, d], in 32 bits."""
    rot = s["rot"]
    y = x.float()
    if s["halves"]:
        y = y.unflatten(2, (2, -1)).flatten(1, 2)
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(dim=-1, keepdim=True) + EPS) * weight
    cs = s["cos_sin"][pos][:, None, :]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    r, rest = y[..., :rot], y[..., rot:]
    if s["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([r, rest], dim=-1).view(x.shape)


def _finish(o1, o2, lam, weight):
    """o1 - lam o2 [..., Hq, d], normalised where there is a weight."""
    o = o1 - lam[..., None] * o2
    if weight is not None:
        o = o * torch.rsqrt(o.square().mean(dim=-1, keepdim=True) + EPS) * weight
    return o.to(BF16)


def _maps(q, k, v, scale, hidden):
    """Both maps of queries q [.., G, T, d] on keys and values [.., L, d] of
    their KV head: ([outputs [.., G, T, d]], [lse [.., G, T]]), in 32 bits."""
    half = q.shape[-1] // 2
    G, T = q.shape[-3:-1]
    outs, lses = [], []
    for qh, kh in ((q[..., :half], k[..., :half]), (q[..., half:], k[..., half:])):
        sc = torch.matmul(qh.flatten(-3, -2), kh.transpose(-2, -1)).mul_(scale)
        sc = sc.unflatten(-2, (G, T)).masked_fill_(hidden, -math.inf)
        m = sc.amax(dim=-1, keepdim=True)
        p = sc.sub_(m).exp_()
        l = p.sum(dim=-1, keepdim=True)
        outs.append(torch.matmul(p.flatten(-3, -2), v).unflatten(-2, (G, T)) / l)
        lses.append((m + l.log()).squeeze(-1))
    return outs, lses


def _plain_decode(s):
    """All sequences at once, padded to the longest."""
    B, Hq, Hkv, d, L = s["B"], s["Hq"], s["Hkv"], s["d"], s["most"]
    G = Hq // Hkv
    k, v = s["k"], s["v"]
    if s["paged"]:
        ids = s["table"].clamp(min=0).long()
        k, v = (x[ids].transpose(1, 2).reshape(B, Hkv, -1, d)[:, :, :L] for x in (k, v))
    hidden = (torch.arange(L, device=k.device)[None, :] >= s["lens"][:, None])[:, None, None, None, :]
    q = s["q"].float().view(B, Hkv, G, 1, d)
    outs, lses = _maps(q, k.float(), v.float(), s["scale"], hidden)
    o1, o2 = (o.reshape(B, Hq, d) for o in outs)
    return _finish(o1, o2, s["lam"], s["weight"]), torch.stack([x.reshape(B, Hq) for x in lses], dim=-1)


def _plain_prompts(s):
    """One sequence after the other, its queries in blocks, each over the keys
    that its last one sees."""
    Hq, Hkv, d = s["Hq"], s["Hkv"], s["d"]
    G = Hq // Hkv
    outs, lses, at = [], [], 0
    for b, n in enumerate(s["new"]):
        L = n + s["ctx"][b]
        k, v = (_tokens(s, x, b, at, L).float().transpose(0, 1) for x in (s["k"], s["v"]))
        q = s["q"][at:at + n].float().view(n, Hkv, G, d).permute(1, 2, 0, 3)
        step = max(1, min(n, (1 << 28) // max(1, Hq * L)))
        for t in range(0, n, step):
            m = min(step, n - t)
            hi = L - n + t + m
            row = torch.arange(m, device=q.device)[:, None] + (L - n + t)
            hidden = torch.arange(hi, device=q.device)[None, :] > row
            o, z = _maps(q[:, :, t:t + m], k[:, :hi], v[:, :hi], s["scale"], hidden)
            o1, o2 = (x.permute(2, 0, 1, 3).reshape(m, Hq, d) for x in o)
            lam = s["lam"][at + t:at + t + m] if s["per_token"] else s["lam"]
            outs.append(_finish(o1, o2, lam, s["weight"]))
            lses.append(torch.stack([x.permute(2, 0, 1).reshape(m, Hq) for x in z], dim=-1))
        at += n
    return torch.cat(outs), torch.cat(lses)


def _tokens(s, x, b, at, L):
    """All keys or values of sequence b, [L, Hkv, d]."""
    if s["paged"]:
        got = x[s["table"][b, :-(-L // PAGE)].long()]
        return got.transpose(1, 2).flatten(0, 1)[:L]
    return x[at:at + L]


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    if work(case)["flops"] > 5e12:
        return None  # over half a minute in 64 bits
    s = prepare(case, seed)
    if s["op"] in ("norm_rope", "append_rope"):
        return _exact_rope(s)
    Hq, Hkv, d = s["Hq"], s["Hkv"], s["d"]
    h2, T = d // 2, s["q"].shape[0]
    out = torch.zeros((T, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, Hq, 2), dtype=torch.float64, device="cuda")
    lam = s["lam"].double().expand(T, Hq)
    at = 0
    for b in range(s["B"]):
        L = s["new"][b] + s["ctx"][b]
        n = 1 if s["op"] == "diff_decode" else s["new"][b]
        for j in range(Hq):
            h = j // (Hq // Hkv)
            if s["paged"]:
                ids = s["table"][b, :-(-L // PAGE)].long()
                k, v = (s[x][ids, h].reshape(-1, d)[:L].double() for x in "kv")
            elif s["op"] == "diff_decode":
                k, v = (s[x][b, h, :L].double() for x in "kv")
            else:
                k, v = (s[x][at:at + L, h].double() for x in "kv")
            for t in range(0, n, 4096):
                rows = slice(at + t, at + min(n, t + 4096))
                q = s["q"][rows, j].double()
                for i in (0, 1):
                    part = slice(i * h2, (i + 1) * h2)
                    sc = q[:, part] @ k[:, part].T * s["scale"]
                    sc += torch.full_like(sc, -math.inf).triu(L - n + t + 1)
                    z = torch.logsumexp(sc, dim=1)
                    lse[rows, j, i] = z
                    o = torch.exp(sc - z[:, None]) @ v
                    out[rows, j] += -lam[rows, j, None] * o if i else o
        at += n
    if s["weight"] is not None:
        out = out / torch.sqrt((out * out).sum(-1, keepdim=True) / d + EPS) * s["weight"].double()
    return out, lse


def _exact_rope(s):
    """The rotation as a product with a complex number of modulus 1 per pair."""
    T, d, rot = s["qkv"].shape[0], s["d"], s["rot"]
    dh = d // 2 if s["halves"] else d
    table = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None, None, :]
    first = torch.arange(0, rot, 2, device="cuda") if s["interleaved"] else torch.arange(rot // 2, device="cuda")
    second = first + (1 if s["interleaved"] else rot // 2)
    at = {"q": (0, s["Hq"]), "k": (s["Hq"], s["Hkv"]), "v": (s["Hq"] + s["Hkv"], s["Hkv"])}
    done = {}
    for n, (h0, H) in at.items():
        x = s["qkv"][:, h0:h0 + H].double().reshape(T, H, d // dh, dh)
        if n != "v":
            if s[n + "_weight"] is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / dh + EPS) * s[n + "_weight"].double()
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
        done[n] = x.reshape(T, H, d)
    if s["op"] == "norm_rope":
        return done["q"], done["k"]
    got = [done["q"]]
    for n in "kv":
        x = done[n].transpose(0, 1)  # [Hkv, T, d]
        Hkv, pool = x.shape[0], s[n + "_pages"].shape[0] * PAGE
        rows = torch.zeros((Hkv, pool, d), dtype=torch.float64, device="cuda")
        if s["fp8"]:
            top = x.abs().amax(dim=2)
            y = x * torch.where(top > 0, 448.0 / top, 0.0)[..., None]
            # e4m3: steps of an eighth of the power of two below, of 2^-9 under 2^-6
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            rows[:, s["slots"]] = torch.round(y / step) * step
            scales = torch.zeros((Hkv, pool), dtype=torch.float64, device="cuda")
            scales[:, s["slots"]] = top / 448
            got += [rows.view(Hkv, -1, PAGE, d).transpose(0, 1), scales.view(Hkv, -1, PAGE).transpose(0, 1)]
        else:
            rows[:, s["slots"]] = x
            got.append(rows.view(Hkv, -1, PAGE, d).transpose(0, 1))
    return tuple(got)
