"""Cases of the cache operators around the verify step: the verifier's attention over the cache, the commit of an
accepted path into a quantised cache, and the way back.

Sizes: 4 key/value heads of 128 with 7 query heads each (a hidden size of 3584), 28 layers of K and V planes, 3 to 7
drafts or a 16-node tree a sequence, caches of 2048 positions and longer ones; 64-wide heads beside them.
"""
import math

import torch

own = False

# the 16-node tree that the tree workloads use (wide at the root, narrowing with depth)
TREE16 = [-1, 0, 0, 0, 0, 1, 1, 1, 2, 2, 3, 5, 5, 6, 8, 11]
FP8 = torch.float8_e4m3fn
CODE_MAX = 448.0  # largest e4m3 value
E_MIN, E_MAX = -40, 120  # range of a scale's exponent; its byte is the exponent + 127


def _att(name, B, T, L, fmt="bf16", G=7, H=4, D=128, prefix=0, new=True, tree="chain"):
    return {"name": name, "op": "attention", "B": B, "T": T, "L": L, "fmt": fmt, "G": G, "H": H, "D": D,
            "prefix": prefix, "new": new, "tree": tree}


def listed():
    return [
        # one user, one token: what a plain decode step costs beside the verify
        _att("att_one_token", 1, 1, 1024),
        # the full verify batch: 7 drafts and the root, caches of 2048 positions at all fills
        _att("att_chain_256", 256, 8, 2048),
        # candidate trees over longer contexts
        _att("att_tree_64", 64, 16, 8192, tree="tree16"),
        # the full batch on a quantised cache of twice the length, 5 drafts
        _att("att_chain_e4m3", 256, 6, 4096, fmt="e4m3"),
        # two very long contexts, single tokens already committed
        _att("att_long_e4m3", 2, 1, 131072, fmt="e4m3", new=False),
        # a system prompt of 8192 tokens that 64 sequences share
        _att("att_prefix_64", 64, 8, 512, prefix=8192),
        # the same with trees on a quantised cache
        _att("att_prefix_tree_e4m3", 128, 16, 256, fmt="e4m3", prefix=2048, tree="tree16"),
        # a smaller model's narrow heads, odd batch, lengths and group, a tree of its own for each sequence
        _att("att_narrow_odd", 37, 5, 3001, G=3, H=5, D=64, tree="random"),
        # one sequence's accepted drafts, every layer
        {"name": "commit_one", "op": "commit", "P": 56, "B": 1, "T": 8, "L": 2048, "H": 4, "D": 128, "path": False},
        # the full batch's accepted tree paths, every layer
        {"name": "commit_tree_256", "op": "commit", "P": 56, "B": 256, "T": 16, "L": 64, "H": 4, "D": 128, "path": True},
        # one layer's K and V of one sequence read back
        {"name": "read_one", "op": "read", "P": 2, "B": 1, "L": 1500, "H": 4, "D": 128},
        # every layer of some sequences, handed to an engine that keeps its cache in bf16
        {"name": "read_layers", "op": "read", "P": 56, "B": 8, "L": 2048, "H": 4, "D": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention"] * 4 + ["commit", "read"])
    D, H = rng.choice([64, 128, 128]), rng.randint(1, 8)
    if op == "commit":
        P, B = 2 * rng.randint(1, 28), _log(rng, 1, 256)
        T = rng.randint(2, 16)
        return {"op": op, "P": P, "B": B, "T": T, "L": T + rng.randint(1, 48), "H": min(H, 4), "D": D, "path": rng.random() < 0.5}
    if op == "read":
        P, B = 2 * rng.randint(1, 28), rng.randint(1, 8)
        return {"op": op, "P": P, "B": B, "L": _log(rng, 16, 2048), "H": min(H, 4), "D": D}
    T, G = _log(rng, 1, 64), rng.randint(1, 8)
    new = T > 1 or rng.random() < 0.5
    B = _log(rng, 1, 256)
    prefix = _log(rng, 64, 8192) if rng.random() < 0.4 else 0
    # no more keys, scores or products than the largest listed cases have
    room = min((1 << 20) * 4 * 128 // (H * D), 256 * 28 * 8 * 2048 // (T * G * H)) // B
    if prefix:
        prefix = max(64, min(prefix, 64 * 28 * 8 * 8192 // (T * G * H * B)))
        room = min(room, 2048)
    L = T + _log(rng, 16, max(32, min(room, 131072)))
    return {"op": op, "B": B, "T": T, "L": L, "fmt": rng.choice(["bf16", "e4m3"]), "G": G, "H": H, "D": D,
            "prefix": prefix, "new": new, "tree": rng.choice(["chain", "random"]) if new else "chain"}


# ---- inputs --------------------------------------------------------------------------------------------------------

def _scale_exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within the scales' range: amax = m * 2^x with m in [0.5, 1)."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 9 + (m > CODE_MAX / 512.0).int(), E_MIN).clamp(E_MIN, E_MAX)


def _power(e):
    """2^e of whole e in -126 .. 127, in 32 bits, exact."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """Codes and scale bytes of rows x [..., D]."""
    x = x.float()
    e = _scale_exponent(x.abs().amax(-1))
    codes = (x * _power(-e)[..., None]).clamp(-CODE_MAX, CODE_MAX).to(FP8)
    return codes, (e + 127).to(torch.uint8)


def _rows(g, dev, *shape):
    """Keys or values of some tokens: normal, the channels of unlike size, as projections leave them."""
    x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
    return x.mul_(torch.linspace(0.5, 1.5, shape[-1], device=dev).to(torch.bfloat16))


class _State:
    pass


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = _State()
    s.op, s.case = case["op"], case
    H, D, B, L = case["H"], case["D"], case["B"], case["L"]
    if s.op == "attention":
        T, fp8 = case["T"], case["fmt"] == "e4m3"
        s.q = torch.randn((B, T, H * case["G"], D), generator=g, device=dev, dtype=torch.bfloat16)
        s.k, s.v = _rows(g, dev, B, L, H, D), _rows(g, dev, B, L, H, D)
        s.ks = s.vs = s.pk = s.pv = s.pks = s.pvs = s.kn = s.vn = s.parent = None
        if fp8:
            s.k, s.ks = _quantise(s.k)
            s.v, s.vs = _quantise(s.v)
        if case["prefix"]:
            s.pk, s.pv = _rows(g, dev, case["prefix"], H, D), _rows(g, dev, case["prefix"], H, D)
            if fp8:
                s.pk, s.pks = _quantise(s.pk)
                s.pv, s.pvs = _quantise(s.pv)
        # lengths at all fills, room for this step's tokens left
        s.len = torch.randint(1, max(2, L - T + 1), (B,), generator=g, device=dev, dtype=torch.int32)
        if case["new"]:
            s.kn, s.vn = _rows(g, dev, B, T, H, D), _rows(g, dev, B, T, H, D)
            if case["tree"] == "tree16":
                s.parent = torch.tensor(TREE16, dtype=torch.int32, device=dev).repeat(B, 1)
            elif case["tree"] == "random":
                n = torch.arange(T, device=dev)
                s.parent = ((torch.rand((B, T), generator=g, device=dev) * n).int().clamp(max=n - 1)).int()
                s.parent[:, 0] = -1
        s.scale = 1.0 / math.sqrt(D)
        s.lse = torch.empty((B, T, H * case["G"]), device=dev) if own else None
    elif s.op == "commit":
        P, T = case["P"], case["T"]
        s.new = _rows(g, dev, P, B, T, H, D)
        s.cache = torch.zeros((P, B, L, H, D), device=dev, dtype=torch.uint8).view(FP8)
        s.scales = torch.zeros((P, B, L, H), device=dev, dtype=torch.uint8)
        s.len = torch.randint(0, L - T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        s.out_len = torch.empty_like(s.len)
        # drafts accepted one after another with probability 0.7, as the verify step leaves them
        ok = (torch.rand((B, T - 1), generator=g, device=dev) < 0.7).int()
        s.acc = ok.cumprod(1).sum(1).int()
        s.path = None
        if case["path"]:  # ascending nodes of a tree whose root is row 0
            order = torch.rand((B, T - 1), generator=g, device=dev).argsort(1) + 1
            keep = torch.arange(T - 1, device=dev) < s.acc[:, None]
            nodes = torch.where(keep, order, T).sort(1).values
            s.path = torch.full((B, T), -1, device=dev, dtype=torch.int32)
            s.path[:, : T - 1] = torch.where(keep, nodes, -1)
    else:
        P = case["P"]
        s.cache, s.scales = _quantise(_rows(g, dev, P, B, L, H, D))
        s.len = torch.randint(1, L + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        s.out = torch.zeros((P, B, L, H, D), device=dev, dtype=torch.bfloat16)
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(s):
    return {"attention": _run_attention, "commit": _run_commit, "read": _run_read}[s.op](s)


def _values(codes, scales):
    """What a cache stands for, in 32 bits."""
    x = codes.float()
    return x if scales is None else x * _power(scales.int() - 127)[..., None]


def _visible(parent, T, dev):
    """[B or 1, T, T]: new token j is i's ancestor or i itself."""
    if parent is None:
        return torch.ones((T, T), dtype=torch.bool, device=dev).tril()[None]
    eye = torch.eye(T, dtype=torch.float32, device=dev)
    up = (parent[:, :, None] == torch.arange(T, device=dev)).float() + eye
    reach = up
    for _ in range(max(1, (T - 1).bit_length())):  # paths of doubling length
        reach = ((reach @ reach) > 0).float()
    return reach > 0


def _run_attention(s):
    if own:
        import speculative_decoding_verification_49_gb300 as sv
        out = sv.verify_attention(s.q, s.k, s.v, s.len, k_new=s.kn, v_new=s.vn, parent=s.parent, k_prefix=s.pk,
                                  v_prefix=s.pv, k_scale=s.ks, v_scale=s.vs, k_prefix_scale=s.pks,
                                  v_prefix_scale=s.pvs, scale=s.scale, lse=s.lse)
        return [out, s.lse]
    c = s.case
    B, T, H, G, D, L = c["B"], c["T"], c["H"], c["G"], c["D"], c["L"]
    dev = s.q.device
    q = s.q.float().view(B, T, H, G, D) * s.scale
    inside = torch.arange(L, device=dev) < s.len[:, None]
    kc = _values(s.k, s.ks)
    vc = _values(s.v, s.vs).masked_fill(~inside[:, :, None, None], 0.0)
    x = [torch.einsum("bthgd,blhd->bhgtl", q, kc).masked_fill(~inside[:, None, None, None], -math.inf)]
    del kc
    if s.pk is not None:
        x.append(torch.einsum("bthgd,lhd->bhgtl", q, _values(s.pk, s.pks)))
    if s.kn is not None:
        seen = _visible(s.parent, T, dev)
        x.append(torch.einsum("bthgd,blhd->bhgtl", q, s.kn.float()).masked_fill(~seen[:, None, None], -math.inf))
    m = x[0].amax(-1)
    for y in x[1:]:
        m = torch.maximum(m, y.amax(-1))
    x = [torch.exp(y - m[..., None]) for y in x]
    total = sum(y.sum(-1) for y in x)
    o = torch.einsum("bhgtl,blhd->bhgtd", x[0], vc)
    if s.pk is not None:
        o += torch.einsum("bhgtl,lhd->bhgtd", x[1], _values(s.pv, s.pvs))
    if s.kn is not None:
        o += torch.einsum("bhgtl,blhd->bhgtd", x[-1], s.vn.float())
    o = (o / total[..., None]).permute(0, 3, 1, 2, 4).reshape(B, T, H * G, D).bfloat16()
    lse = (m + total.log()).permute(0, 3, 1, 2).reshape(B, T, H * G)
    return [o, lse]


def _run_commit(s):
    if own:
        import speculative_decoding_verification_49_gb300 as sv
        sv.kv_commit_path(s.new, s.cache, s.len, s.acc, path=s.path, lead=1, scale=s.scales, out_len=s.out_len)
        return [s.cache, s.scales, s.out_len]
    B, T = s.case["B"], s.case["T"]
    i = torch.arange(T, device=s.new.device)
    row = i.expand(B, T) if s.path is None else torch.cat([torch.zeros_like(s.path[:, :1]), s.path[:, :-1]], 1)
    b, i = (i <= s.acc[:, None]).nonzero(as_tuple=True)
    codes, scales = _quantise(s.new[:, b, row[b, i].long()])
    at = s.len.long()[b] + i
    s.cache.view(torch.uint8)[:, b, at] = codes.view(torch.uint8)
    s.scales[:, b, at] = scales
    return [s.cache, s.scales, s.len + 1 + s.acc]


def _run_read(s):
    if own:
        import speculative_decoding_verification_49_gb300 as sv
        sv.kv_read(s.cache, s.scales, s.len, out=s.out)
        return [s.out]
    inside = torch.arange(s.case["L"], device=s.out.device) < s.len[:, None]
    s.out.copy_(torch.where(inside[None, :, :, None, None], _values(s.cache, s.scales), 0.0))
    return [s.out]


# ---- what a pass cannot do without -----------------------------------------------------------------------------------

def work(case):
    H, D, B, L = case["H"], case["D"], case["B"], case["L"]
    if case["op"] == "attention":
        T, R = case["T"], case["T"] * case["G"] * H
        token = H * (2 * D * 2 if case["fmt"] == "bf16" else 2 * (D + 1))
        keys = B * (1 + max(1, L - T)) / 2
        new = B * T * H * D * 4 if case["new"] else 0
        pairs = R * (keys + B * case["prefix"]) + (B * R * (T + 1) / 2 if case["new"] else 0)
        return {"bytes": (keys + case["prefix"]) * token + new + B * R * (D * 4 + 4), "flops": 4 * D * pairs}
    if case["op"] == "commit":
        rows = case["P"] * B * (1 + sum(0.7 ** k for k in range(1, case["T"])))
        return {"bytes": rows * H * (2 * D + D + 1), "flops": 2 * rows * H * D}
    rows = case["P"] * B * (L + 1) / 2
    return {"bytes": rows * H * (3 * D + 1), "flops": rows * H * D}


# ---- the same in 64 bits, from the definitions -----------------------------------------------------------------------

def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _code_values64(x):
    """Nearest e4m3 value of |x| <= 448, ties to the even code: steps of 2^(k-3) in [2^k, 2^(k+1)), of 2^-9 below 2^-6."""
    k = (torch.frexp(x.abs())[1] - 1).clamp(min=-6)
    step = _power64(k - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if s.op == "attention":
        return _exact_attention(s)
    if s.op == "commit":
        T, cache = case["T"], torch.zeros(s.cache.shape, dtype=torch.float64, device=s.cache.device)
        scales = torch.zeros_like(s.scales)
        for b, (n, a) in enumerate(zip(s.len.tolist(), s.acc.tolist())):
            rows = [0] + (list(range(1, a + 1)) if s.path is None else s.path[b, :a].tolist())
            x = s.new[:, b, rows].double()
            amax = x.abs().amax(-1)
            e = torch.ceil(torch.log2(amax / CODE_MAX)).clamp(E_MIN, E_MAX)
            e = torch.where((e > E_MIN) & (amax <= CODE_MAX * _power64(e - 1)), e - 1, e)  # a logarithm just above a whole number
            cache[:, b, n : n + a + 1] = _code_values64(x * _power64(-e)[..., None])
            scales[:, b, n : n + a + 1] = (e + 127).to(torch.uint8)
        return [cache, scales, s.len + s.acc + 1]
    out = torch.zeros(s.out.shape, dtype=torch.float64, device=s.out.device)
    for b, n in enumerate(s.len.tolist()):
        out[:, b, :n] = s.cache[:, b, :n].double() * _power64(s.scales[:, b, :n].int() - 127)[..., None]
    return [out]


def _exact_attention(s):
    c = s.case
    B, T, H, G, D = c["B"], c["T"], c["H"], c["G"], c["D"]

    def whole(x, scales):
        return x.double() if scales is None else x.double() * _power64(scales.int() - 127)[..., None]

    out = torch.empty((B, T, H, G, D), dtype=torch.float64, device=s.q.device)
    lse = torch.empty((B, T, H, G), dtype=torch.float64, device=s.q.device)
    parents = s.parent.tolist() if s.parent is not None else [[j - 1 for j in range(T)]] * B
    pk, pv = (whole(s.pk, s.pks), whole(s.pv, s.pvs)) if s.pk is not None else (None, None)
    for b, n in enumerate(s.len.tolist()):
        keys = [whole(s.k[b, :n], s.ks[b, :n] if s.ks is not None else None)]
        vals = [whole(s.v[b, :n], s.vs[b, :n] if s.vs is not None else None)]
        if pk is not None:
            keys.insert(0, pk)
            vals.insert(0, pv)
        if s.kn is not None:
            keys.append(s.kn[b].double())
            vals.append(s.vn[b].double())
        k, v = torch.cat(keys), torch.cat(vals)
        x = (s.q[b].double().view(T, H, G, D).permute(1, 0, 2, 3).reshape(H, T * G, D) @ k.permute(1, 2, 0)) * s.scale
        if s.kn is not None:
            hide = torch.ones((T, T), dtype=torch.bool)
            for t in range(T):
                j = t
                while j >= 0:
                    hide[t, j] = False
                    j = parents[b][j]
            x.view(H, T, G, -1)[..., k.shape[0] - T :].masked_fill_(hide.to(x.device)[None, :, None], -math.inf)
        lse[b] = torch.logsumexp(x, -1).view(H, T, G).permute(1, 0, 2)
        out[b] = (torch.softmax(x, -1) @ v.permute(1, 0, 2)).view(H, T, G, D).permute(1, 0, 2, 3)
    return [out.reshape(B, T, H * G, D), lse.reshape(B, T, H * G)]
