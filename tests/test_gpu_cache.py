"""The cache operators on the GPU against plain 64-bit references (needs a GB300)."""
import math

import numpy as np
import pytest
import torch

import cacheref as ref
import speculative_decoding_verification_49_gb300 as sv

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_49_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _bf(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def _cuda(t):
    return None if t is None else t.cuda()


def _byte_equal(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


# ---- commit ----------------------------------------------------------------------------------------------------

def _commit_case(g, P, B, T, H, D, L, fmt, tree, lead):
    rows = _bf(g, P, B, T, H, D)
    rows *= torch.exp2(torch.randint(-12, 13, (P, B, T, H, 1), generator=g).float()).to(torch.bfloat16)
    acc = torch.randint(0, T - lead + 1, (B,), generator=g, dtype=torch.int32)
    lens = torch.tensor([int(torch.randint(0, L - lead - int(a) + 1, (1,), generator=g)) for a in acc], dtype=torch.int32)
    path = None
    if tree:
        path = torch.full((B, T), -1, dtype=torch.int32)
        for b in range(B):
            nodes = (torch.randperm(T - lead, generator=g)[: int(acc[b])] + lead).sort().values
            path[b, : int(acc[b])] = nodes.int()
    dt = FP8 if fmt == "e4m3" else torch.bfloat16
    cache = torch.randint(0, 256, (P, B, L, H, D * (1 if dt == FP8 else 2)), generator=g, dtype=torch.uint8).view(dt)
    scale = torch.randint(1, 255, (P, B, L, H), generator=g, dtype=torch.uint8) if dt == FP8 else None
    return rows, cache, scale, lens, acc, path


def _commit_want(rows, cache, scale, lens, acc, path, lead):
    cache, lens = cache.clone(), lens.clone()
    scale = None if scale is None else scale.clone()
    T, L = rows.shape[2], cache.shape[2]
    bits = 0
    for b in range(rows.shape[1]):
        a, n = int(acc[b]), int(lens[b])
        if a < 0:
            continue
        src = list(range(lead)) + [int(path[b, i]) if path is not None and i < path.shape[1] else lead + i
                                   for i in range(a)]
        if lead + a > T:
            bits |= sv.SV_KV_BAD_COUNT
        elif n < 0 or n + lead + a > L:
            bits |= sv.SV_KV_OVERFLOW
        elif any(not 0 <= r < T for r in src):
            bits |= sv.SV_KV_BAD_PATH
        else:
            x = rows[:, b, src]
            if scale is not None:
                codes, s = ref.quantise(x)
                cache[:, b, n:n + lead + a] = codes
                scale[:, b, n:n + lead + a] = s
                if not torch.isfinite(x.float()).all():
                    bits |= sv.SV_KV_NONFINITE
            else:
                cache[:, b, n:n + lead + a] = x
            lens[b] = n + lead + a
    return cache, scale, lens, bits


def _commit_gpu(rows, cache, scale, lens, acc, path, lead, in_place=True):
    c, s, ln = cache.cuda(), _cuda(scale), lens.cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = None if in_place else torch.full_like(ln, -7)
    got = sv.kv_commit_path(rows.cuda(), c, ln, acc.cuda(), path=_cuda(path), lead=lead, scale=s, out_len=out, status=st)
    torch.cuda.synchronize()
    if not in_place:
        assert torch.equal(ln.cpu(), lens)
    return c.cpu(), None if s is None else s.cpu(), got.cpu(), int(st)


def _check_commit(case, lead, in_place=True):
    want = _commit_want(*case, lead)
    got = _commit_gpu(*case, lead, in_place)
    assert _byte_equal(got[0], want[0])
    assert want[1] is None or torch.equal(got[1], want[1])
    assert torch.equal(got[2], want[2]) and got[3] == want[3]


@pytest.mark.parametrize("P,B,T,H,D,L,lead", [
    (1, 1, 1, 1, 16, 1, 0), (2, 3, 8, 4, 128, 20, 1), (3, 5, 4, 2, 64, 9, 1), (5, 7, 6, 3, 80, 11, 0),
    (2, 4, 16, 1, 256, 40, 1), (4, 33, 5, 5, 48, 30, 2), (56, 9, 8, 4, 128, 64, 1), (2, 300, 3, 1, 32, 6, 1)])
@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("tree", [False, True])
def test_commit_path_matches_the_reference(P, B, T, H, D, L, lead, fmt, tree):
    case = _commit_case(_gen(P * 31 + B), P, B, T, H, D, L, fmt, tree, lead)
    _check_commit(case, lead, in_place=B % 2 == 1)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
def test_commit_path_bad_sequences_leave_everything(fmt):
    rows, cache, scale, lens, acc, path = _commit_case(_gen(3), 3, 8, 6, 2, 64, 12, fmt, True, 1)
    acc[0] = -1                      # the verify flagged it
    acc[1] = 6                       # lead + 6 > T
    lens[2] = 12 - int(acc[2])       # one row too many with the lead
    lens[3] = -2
    acc[4], path[4, 0] = 2, 6        # past the scratch
    acc[5], path[5, 1] = 2, -1
    lens[4] = lens[5] = 0
    lens[6] = 2 ** 31 - 1            # the sum would pass 32 bits
    _check_commit((rows, cache, scale, lens, acc, path), 1)


def test_commit_path_values_at_the_edges():
    """Zero rows, exact powers, halfway cases, subnormal codes, the largest and smallest magnitudes, NaN and infinities."""
    g = _gen(4)
    x = torch.zeros((1, 1, 16, 1, 64), dtype=torch.bfloat16)
    x[0, 0, 1, 0, 0] = 448.0
    x[0, 0, 2, 0, 0] = 450.0                                  # the next bf16 above 448 * 2^0
    x[0, 0, 3] = torch.linspace(0, 448, 64).to(torch.bfloat16)
    x[0, 0, 4] = (torch.arange(64) * 2.0 ** -10 + 0.0).to(torch.bfloat16)
    x[0, 0, 4, 0, 63] = 448.0
    x[0, 0, 5, 0, :] = torch.finfo(torch.bfloat16).max
    x[0, 0, 6, 0, :] = 1e-30
    x[0, 0, 7, 0, :] = 2.0 ** -133                            # smallest subnormal
    x[0, 0, 8] = _bf(g, 1, 64)
    x[0, 0, 8, 0, 3] = math.inf
    x[0, 0, 9] = _bf(g, 1, 64)
    x[0, 0, 9, 0, 5] = math.nan
    x[0, 0, 9, 0, 6] = -math.inf
    x[0, 0, 10, 0, :] = math.nan
    x[0, 0, 11] = torch.arange(-32, 32).float() * 17          # ties of 4-bit significands
    x[0, 0, 12] = -x[0, 0, 3]
    x[0, 0, 13, 0, :] = -0.0
    cache = torch.zeros((1, 1, 16, 1, 64), dtype=torch.uint8).view(FP8)
    scale = torch.zeros((1, 1, 16, 1), dtype=torch.uint8)
    _check_commit((x, cache, scale, torch.zeros(1, dtype=torch.int32), torch.full((1,), 16, dtype=torch.int32), None), 0)


# ---- read-back ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("P,B,H,D,L,rows,start", [
    (1, 1, 1, 16, 1, None, False), (2, 3, 4, 128, 50, None, False), (3, 4, 2, 64, 33, 20, True),
    (5, 2, 3, 80, 17, 17, True), (2, 2, 1, 256, 9, 30, False), (56, 3, 4, 128, 40, 8, True)])
def test_read_matches_the_reference(P, B, H, D, L, rows, start):
    g = _gen(P + L)
    cache = torch.randint(0, 256, (P, B, L, H, D), generator=g, dtype=torch.uint8).view(FP8)
    scale = torch.randint(87, 248, (P, B, L, H), generator=g, dtype=torch.uint8)
    lens = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
    lens[0] = L
    st = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32) if start else None
    n = L if rows is None else rows
    out = _bf(g, P, B, n, H, D)
    want = out.clone()
    v = ref.values(cache, scale)
    for b in range(B):
        s0 = 0 if st is None else int(st[b])
        k = max(0, min(int(lens[b]) - s0, n))
        want[:, b, :k] = v[:, b, s0:s0 + k].to(torch.bfloat16)
    got = sv.kv_read(cache.cuda(), scale.cuda(), lens.cuda(), start=_cuda(st), rows=rows, out=out.cuda()).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))


def test_read_bad_lengths_are_flagged_and_skipped():
    cache = torch.zeros((2, 4, 5, 1, 16), dtype=torch.uint8).view(FP8).cuda()
    scale = torch.full((2, 4, 5, 1), 127, dtype=torch.uint8, device="cuda")
    lens = torch.tensor([6, -1, 5, 3], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 0, -1, 4], dtype=torch.int32, device="cuda")
    out = torch.full((2, 4, 5, 1, 16), 9.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.kv_read(cache, scale, lens, start=start, out=out, status=st)
    assert int(st) == sv.SV_KV_OVERFLOW and bool((out == 9).all())


# ---- attention -----------------------------------------------------------------------------------------------------

def _attention_case(seed, B, T, H, G, D, L, fmt="bf16", prefix=0, new=True, tree=False, lens=None):
    g = _gen(seed)
    c = dict(q=_bf(g, B, T, H * G, D), k=_bf(g, B, L, H, D), v=_bf(g, B, L, H, D))
    if lens is None:
        lens = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
    c["lens"] = torch.as_tensor(lens, dtype=torch.int32)
    c["k_new"] = _bf(g, B, T, H, D) if new else None
    c["v_new"] = _bf(g, B, T, H, D) if new else None
    c["parent"] = None
    if tree and new:
        c["parent"] = torch.stack([(torch.rand(B, generator=g) * n).int().clamp(max=n - 1) for n in range(T)], 1).int()
        c["parent"][:, 0] = -1
    c["k_prefix"] = _bf(g, prefix, H, D) if prefix else None
    c["v_prefix"] = _bf(g, prefix, H, D) if prefix else None
    c["ks"] = c["vs"] = c["kps"] = c["vps"] = None
    if fmt == "e4m3":
        c["k"], c["ks"] = ref.quantise(c["k"])
        c["v"], c["vs"] = ref.quantise(c["v"])
        if prefix:
            c["k_prefix"], c["kps"] = ref.quantise(c["k_prefix"])
            c["v_prefix"], c["vps"] = ref.quantise(c["v_prefix"])
    return c


def _attention_gpu(c, scale=None, **more):
    B, T, Hq, _ = c["q"].shape
    lse = torch.full((B, T, Hq), -77.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = sv.verify_attention(_cuda(c["q"]), _cuda(c["k"]), _cuda(c["v"]), _cuda(c["lens"]), k_new=_cuda(c["k_new"]),
                              v_new=_cuda(c["v_new"]), parent=_cuda(c["parent"]), k_prefix=_cuda(c["k_prefix"]),
                              v_prefix=_cuda(c["v_prefix"]), k_scale=_cuda(c["ks"]), v_scale=_cuda(c["vs"]),
                              k_prefix_scale=_cuda(c["kps"]), v_prefix_scale=_cuda(c["vps"]), scale=scale, lse=lse,
                              status=st, **more)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), int(st)


def _check_attention(c, scale=None):
    out, lse, st = _attention_gpu(c, scale)
    assert st == 0
    o, ll, tol, tol_lse = ref.attention(c["q"], c["k"], c["v"], c["lens"], c["k_new"], c["v_new"], c["parent"],
                                        c["k_prefix"], c["v_prefix"], c["ks"], c["vs"], c["kps"], c["vps"], scale)
    ref.assert_close(out, o, tol, "out")
    ref.assert_close(lse, ll, tol_lse, "lse")


SHAPES = [
    # B, T, H, G, D, L, prefix, new, tree
    (1, 1, 1, 1, 128, 1, 0, True, False), (1, 1, 4, 7, 128, 1024, 0, True, False), (2, 1, 2, 1, 64, 300, 0, False, False),
    (3, 8, 4, 7, 128, 513, 0, True, False), (2, 16, 2, 8, 128, 200, 0, True, True), (5, 5, 3, 3, 64, 129, 0, True, True),
    (2, 37, 1, 7, 128, 260, 0, True, True), (1, 128, 1, 8, 64, 70, 0, True, True), (2, 128, 2, 1, 128, 257, 0, True, False),
    (4, 3, 1, 5, 128, 127, 100, True, True), (7, 8, 2, 7, 128, 64, 700, True, False), (9, 16, 1, 7, 64, 33, 129, True, True),
    (3, 1, 2, 4, 128, 40, 1, False, False), (33, 2, 5, 2, 64, 31, 256, True, True), (2, 4, 2, 2, 128, 5000, 0, True, True),
    (40, 8, 1, 7, 128, 2, 300, True, False), (300, 1, 1, 1, 64, 20, 0, True, False), (1, 2, 1, 3, 128, 40000, 0, True, False),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,T,H,G,D,L,prefix,new,tree", SHAPES)
def test_attention_matches_the_reference(B, T, H, G, D, L, prefix, new, tree, fmt):
    _check_attention(_attention_case(B * 7 + T + L, B, T, H, G, D, L, fmt, prefix, new, tree))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(4, 4), (17, 1), (5, 5), (31, 1), (8, 4), (11, 3), (5, 8), (6, 8), (7, 7), (21, 3), (8, 8),
                                 (13, 5), (9, 14), (16, 8), (43, 3), (32, 8), (37, 7)])
def test_attention_rows_of_a_sequence(T, G, D, fmt):
    """Rows on both sides of every count at which another form takes over, with long and short sequences side by side."""
    lens = [0, 1, 130, 1290, 128, 700, 15, 1291, 256]
    _check_attention(_attention_case(T * G, len(lens), T, 3, G, D, 1291, fmt, new=True, tree=T % 2 == 0, lens=lens))
    _check_attention(_attention_case(T + G, 2, T, 1, G, D, 390, fmt, new=False, lens=[390, 257]))


@pytest.mark.parametrize("B,T,G,L,prefix", [(220, 3, 4, 90, 0), (220, 5, 5, 200, 0), (220, 6, 7, 300, 0), (230, 10, 6, 140, 0),
                                            (60, 3, 4, 300, 300), (130, 5, 6, 129, 128), (90, 9, 5, 40, 1000),
                                            (40, 16, 8, 260, 257)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_many_segments(B, T, G, L, prefix, fmt):
    """More segments than CTAs, most of them short, alone and behind a prefix that has blocks of rows of its own."""
    lens = [(b * 37 + b * b) % (L + 1) for b in range(B)]
    _check_attention(_attention_case(B + T, B, T, 2, G, 128, L, fmt, prefix=prefix, tree=True, lens=lens))


@pytest.mark.parametrize("B,T,H,G,D,L,prefix", [(40, 8, 4, 7, 128, 150, 1100), (41, 5, 5, 3, 64, 129, 2049), (5, 8, 16, 4, 64, 300, 1300),
                                                (3, 16, 17, 5, 128, 64, 1409), (9, 9, 8, 4, 128, 700, 2000)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_long_prefixes(B, T, H, G, D, L, prefix, fmt):
    """Prefixes of so many tiles that each weighs as two of a sequence's, cut at both of its halves."""
    lens = [(b * 41 + b * b) % (L + 1) for b in range(B)]
    _check_attention(_attention_case(B + prefix, B, T, H, G, D, L, fmt, prefix=prefix, tree=T % 2 == 0, lens=lens))


@pytest.mark.parametrize("B,T,H,G,D,L,prefix", [(3, 40, 2, 8, 64, 100, 300), (1, 128, 1, 300, 64, 130, 0), (2, 128, 1, 96, 128, 3, 129),
                                                (600, 1, 1, 1, 128, 5, 1)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_many_rows(B, T, H, G, D, L, prefix, fmt):
    """Sequences of several blocks of rows, and many of one row behind one prefix key."""
    lens = [(b * 41 + L) % (L + 1) for b in range(B)]
    _check_attention(_attention_case(B + G, B, T, H, G, D, L, fmt, prefix=prefix, tree=True, lens=lens))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_of_more_sequences_than_16_bits_count(fmt):
    B, keep = 66000, [0, 1, 2, 1023, 32767, 32768, 65535, 65536, 65998, 65999]
    c = _attention_case(33, B, 1, 1, 2, 64, 3, fmt, lens=[b % 4 for b in range(B)])
    out, lse, st = _attention_gpu(c)
    assert st == 0
    few = {k: (None if v is None else v.view(torch.uint8)[keep].view(FP8) if v.dtype == FP8 else v[keep])
           for k, v in c.items()}
    o, ll, tol, tol_lse = ref.attention(few["q"], few["k"], few["v"], few["lens"], few["k_new"], few["v_new"],
                                        few["parent"], None, None, few["ks"], few["vs"])
    ref.assert_close(out[keep], o, tol, "out")
    ref.assert_close(lse[keep], ll, tol_lse, "lse")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,G", [(2, 4), (5, 5), (3, 13), (16, 5)])
def test_attention_a_row_that_is_not_finite_leaves_the_others(T, G, fmt):
    """NaN and infinities in one query row: every other row's result is what it is without them, bit for bit."""
    c = _attention_case(35, 3, T, 2, G, 128, 500, fmt, tree=True, lens=[500, 130, 7])
    want = _attention_gpu(c)
    for bad in (math.nan, math.inf):
        d = dict(c, q=c["q"].clone())
        d["q"][1, T - 1, G, 5] = bad
        got = _attention_gpu(d)
        rest = torch.ones(want[1].shape, dtype=torch.bool)
        rest[1, T - 1, G] = False
        assert torch.equal(got[0][rest], want[0][rest]) and torch.equal(got[1][rest], want[1][rest])
        if math.isnan(bad):
            assert torch.isnan(got[0][1, T - 1, G].float()).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,H,L", [(1, 1, 1), (1, 2, 1152), (1, 2, 1281), (19, 8, 1152), (51, 3, 130), (152, 1, 1281)])
def test_attention_few_segments_whole_and_cut(B, H, L, fmt):
    """Segment counts and lengths on both sides of those that are not cut."""
    for T, G in ((1, 7), (4, 10), (40, 4)):
        _check_attention(_attention_case(B + L, B, T, H, G, 64, L, fmt, lens=[L - b % 2 for b in range(B)]))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_lengths_at_tile_borders(fmt, D):
    lens = [0, 1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384, 400]
    _check_attention(_attention_case(5, len(lens), 3, 2, 2, D, 400, fmt, lens=lens, tree=True))
    _check_attention(_attention_case(6, len(lens), 1, 2, 2, D, 400, fmt, lens=lens, new=False))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_without_any_key_is_zero(fmt):
    c = _attention_case(8, 3, 2, 2, 3, 128, 20, fmt, new=False, lens=[0, 5, 0])
    out, lse, st = _attention_gpu(c)
    assert st == 0
    assert (out[0] == 0).all() and (out[2] == 0).all() and (lse[0] == -math.inf).all() and (lse[2] == -math.inf).all()
    _check_attention(c)
    # no cache at all: the new tokens alone
    c = _attention_case(9, 3, 6, 2, 3, 64, 0, fmt, tree=True, lens=[0, 0, 0])
    _check_attention(c)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_stale_rows_and_unseen_tokens_do_not_matter(fmt, D):
    """NaN, infinities and NaN codes behind the length and in unseen tokens; a NaN in a seen one."""
    c = _attention_case(11, 4, 6, 2, 3, D, 300, fmt, prefix=130, tree=True, lens=[0, 17, 128, 299])
    want = _attention_gpu(c)
    for b, n in enumerate(c["lens"].tolist()):
        for name in ("k", "v"):
            x = c[name]
            (x.view(torch.uint8) if fmt == "e4m3" else x)[b, n:] = 0x7f if fmt == "e4m3" else math.nan
        if fmt == "e4m3":
            c["ks"][b, n:] = 255
            c["vs"][b, n:] = 255
    got = _attention_gpu(c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # token 5's entry is seen by token 5 alone (it is the last)
    c["v_new"][:, 5, 1, 3] = math.inf
    c["k_new"][:, 5, 0] = math.nan
    got = _attention_gpu(c)
    assert torch.equal(got[0][:, :5], want[0][:, :5]) and torch.equal(got[1][:, :5], want[1][:, :5])
    assert not torch.isfinite(got[0][:, 5].float()).any()


def test_attention_large_scores_and_far_maxima():
    """Scores in the hundreds whose maximum comes late, early, and in the last tile; one key that takes everything."""
    for fmt in ("bf16", "e4m3"):
        c = _attention_case(13, 3, 2, 1, 2, 128, 900, fmt="bf16", lens=[900, 777, 130])
        c["k"] *= 12
        c["q"] *= 3
        c["k"][0, 899] = c["q"][0, 0, 0] * 4
        c["k"][1, 0] = c["q"][1, 1, 1] * 4
        if fmt == "e4m3":
            c["k"], c["ks"] = ref.quantise(c["k"])
            c["v"], c["vs"] = ref.quantise(c["v"])
        _check_attention(c)
        _check_attention(c, scale=0.9)
        _check_attention(c, scale=1e-3)


def test_attention_values_of_unlike_size():
    """Value scales from 2^-30 to 2^20 side by side, and rows of zeros: the sums keep every key's weight."""
    c = _attention_case(14, 2, 3, 2, 2, 128, 700, lens=[700, 300])
    g = _gen(15)
    c["v"] *= torch.exp2(torch.randint(-30, 21, (2, 700, 2, 1), generator=g).float()).to(torch.bfloat16)
    c["v"][:, ::5] = 0
    c["k"], c["ks"] = ref.quantise(c["k"])
    c["v"], c["vs"] = ref.quantise(c["v"])
    _check_attention(c)


def test_attention_one_heavy_key_over_many_light_ones():
    """Half of the mass on one key, the other half on 20000 keys of 2^-15 each, all values positive."""
    for fmt in ("bf16", "e4m3"):
        c = _attention_case(16, 1, 1, 1, 1, 128, 20001, lens=[20001], new=False)
        c["q"][:] = 1.0
        c["k"][:] = 0.0
        c["k"][0, 3] = 0.875 * math.sqrt(128) * math.log(20000) / 128 / 0.875
        c["v"] = c["v"].abs()
        if fmt == "e4m3":
            c["k"], c["ks"] = ref.quantise(c["k"])
            c["v"], c["vs"] = ref.quantise(c["v"])
        _check_attention(c)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_invalid_sequences(fmt):
    c = _attention_case(17, 6, 4, 2, 2, 64, 200, fmt, tree=True, lens=[10, 201, -1, 30, 40, 200])
    c["parent"][3, 2] = 2            # not below itself
    c["parent"][4, 0] = 0            # the root has no parent
    out, lse, st = _attention_gpu(c)
    assert st == sv.SV_ATTN_BAD_LEN | sv.SV_ATTN_BAD_TREE
    for b in (1, 2, 3, 4):
        assert torch.isnan(out[b].float()).all() and torch.isnan(lse[b]).all()
    keep = [0, 5]
    good = {k: (None if v is None else v.view(torch.uint8)[keep].view(FP8) if v.dtype == FP8 else v[keep])
            for k, v in c.items()}
    o, ll, tol, tol_lse = ref.attention(good["q"], good["k"], good["v"], good["lens"], good["k_new"], good["v_new"],
                                        good["parent"], None, None, good["ks"], good["vs"])
    ref.assert_close(out[keep], o, tol, "out")
    ref.assert_close(lse[keep], ll, tol_lse, "lse")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_on_views_of_a_fused_projection(fmt):
    """q, k_new and v_new as views of [B, T, (Hq + 2 H) D], also with sequences and tokens swapped in memory."""
    B, T, H, G, D = 3, 5, 2, 3, 128
    c = _attention_case(19, B, T, H, G, D, 150, fmt, tree=True)
    want = _attention_gpu(c)
    for swap in (False, True):
        flat = torch.cat([c["q"].reshape(B, T, -1), c["k_new"].reshape(B, T, -1), c["v_new"].reshape(B, T, -1)], -1).cuda()
        if swap:
            flat = flat.transpose(0, 1).contiguous().transpose(0, 1)
        q, kn, vn = flat.split([H * G * D, H * D, H * D], -1)
        dev = {k: _cuda(v) for k, v in c.items()}
        lse = torch.empty((B, T, H * G), device="cuda")
        out = sv.verify_attention(q.unflatten(-1, (H * G, D)), dev["k"], dev["v"], dev["lens"],
                                  k_new=kn.unflatten(-1, (H, D)), v_new=vn.unflatten(-1, (H, D)), parent=dev["parent"],
                                  k_scale=dev["ks"], v_scale=dev["vs"], lse=lse)
        assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_repeats_bit_for_bit_and_in_graphs_on_two_streams(fmt):
    """The same call again, captured into two graphs that replay at the same time, and with its stream given."""
    cases = [_attention_case(20 + i, 9, 8, 2, 7, 128, 700, fmt, prefix=300, tree=True) for i in range(2)]
    want = [_attention_gpu(c) for c in cases]
    graphs, outs = [], []
    keep = []
    for c in cases:
        d = {k: _cuda(v) for k, v in c.items()}
        keep.append(d)

        def call(stream=None):
            return sv.verify_attention(d["q"], d["k"], d["v"], d["lens"], k_new=d["k_new"], v_new=d["v_new"],
                                       parent=d["parent"], k_prefix=d["k_prefix"], v_prefix=d["v_prefix"],
                                       k_scale=d["ks"], v_scale=d["vs"], k_prefix_scale=d["kps"],
                                       v_prefix_scale=d["vps"], stream=stream)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want[len(graphs)][0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o.cpu(), w[0])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,G,prefix", [(8, 7, 0), (8, 7, 300), (5, 3, 0), (9, 5, 0), (13, 5, 0)])
def test_attention_does_not_depend_on_what_ran_before(T, G, prefix, fmt):
    """Rows behind a sequence's last one hold what an earlier kernel left in shared memory: the result is the same bit for bit."""
    c = _attention_case(41, 40, T, 2, G, 128, 900, fmt, prefix=prefix, tree=True)
    c["q"] *= 4                      # scores that move the references now and then
    other = [_attention_case(42, 40, 16, 2, 8, 128, 300, "bf16", tree=True) for _ in range(2)]
    other[0]["q"] *= 1000
    other[1]["q"] *= 0
    _attention_gpu(other[1])
    want = _attention_gpu(c)
    for _ in range(3):
        for o in other:
            _attention_gpu(o)
            got = _attention_gpu(c)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_over_a_cache_past_32_bit_offsets():
    """5 GB a plane: the last sequences' rows lie past 2^32 bytes (and 2^31 elements)."""
    B, L, H, D, G, T = 41, 131072, 4, 128, 2, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k = torch.empty((B, L, H, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty((B, L, H, D), dtype=torch.bfloat16, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for b, n in ((0, 70), (39, 300), (40, 131072)):
        k[b, :n].normal_(generator=g)
        v[b, :n].normal_(generator=g)
        lens[b] = n
    q = torch.randn((B, T, H * G, D), generator=g, device="cuda").to(torch.bfloat16)
    out = sv.verify_attention(q, k, v, lens)
    for b, n in ((0, 70), (39, 300), (40, 131072)):
        o, _, tol, _ = ref.attention(q[b:b + 1].cpu(), k[b:b + 1, :n].cpu(), v[b:b + 1, :n].cpu(), [n])
        ref.assert_close(out[b:b + 1], o, tol, f"sequence {b}")
    assert (out[1:39] == 0).all()


def test_front_end_refusals():
    c = _attention_case(23, 2, 3, 2, 2, 64, 40)
    d = {k: _cuda(v) for k, v in c.items()}

    def call(**over):
        a = dict(q=d["q"], k_cache=d["k"], v_cache=d["v"], cache_len=d["lens"], k_new=d["k_new"], v_new=d["v_new"])
        return sv.verify_attention(**{**a, **over})

    for over in (dict(q=d["q"].float()), dict(q=c["q"]), dict(k_cache=d["k"].float()), dict(v_cache=d["v"][:, :20]),
                 dict(cache_len=d["lens"].long()), dict(k_new=None), dict(k_scale=torch.zeros(1, device="cuda")),
                 dict(k_cache=d["k"].to(FP8), v_cache=d["v"].to(FP8)), dict(k_cache=d["k"].transpose(1, 2)),
                 dict(q=d["q"].transpose(2, 3).contiguous().transpose(2, 3)), dict(k_prefix=d["k"][0]),
                 dict(parent=d["lens"]), dict(k_new=None, v_new=None, parent=d["lens"]),
                 dict(out=torch.empty((1,), device="cuda")), dict(lse=torch.empty((2, 3, 4), device="cuda").half())):
        with pytest.raises(ValueError):
            call(**over)
    with pytest.raises(sv.SpecVerifyError):
        call(scale=-1.0)
    rows, cache, scale, lens, acc, _ = (_cuda(t) for t in _commit_case(_gen(1), 2, 2, 3, 2, 64, 9, "e4m3", False, 1))
    for a, k in (((rows.float(), cache, lens, acc), dict(scale=scale)), ((rows, cache, lens, acc), {}),
                 ((rows, cache, lens.long(), acc), dict(scale=scale)), ((rows[:, :1], cache, lens, acc), dict(scale=scale)),
                 ((rows, cache, lens, acc), dict(scale=scale, path=lens))):
        with pytest.raises(ValueError):
            sv.kv_commit_path(*a, **k)
    with pytest.raises(sv.SpecVerifyError):
        sv.kv_commit_path(rows, cache, lens, acc, scale=scale, lead=4)
    with pytest.raises(ValueError):
        sv.kv_read(cache, scale[:1], lens)
    with pytest.raises(ValueError):
        sv.kv_read(cache, scale, lens, out=rows.float())


# ---- together ------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_verify_step_end_to_end(fmt):
    """Attention of a tree over the cache, the tree verify, the commit of the path it accepts, twice in a row; then the
    next step's attention over the cache equals the reference on what was committed, and the read-back its values."""
    B, M, H, G, D, L, V = 4, 9, 2, 3, 64, 64, 512
    T = M + 1
    g = _gen(30)
    dt = FP8 if fmt == "e4m3" else torch.bfloat16
    cache = torch.zeros((2, B, L, H, D * (1 if dt == FP8 else 2)), dtype=torch.uint8).view(dt).cuda()
    scale = torch.zeros((2, B, L, H), dtype=torch.uint8, device="cuda") if dt == FP8 else None
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ctx = sv.SpecVerify(B, M, V, "f32")
    parent = torch.tensor([-1, 0, 0, 1, 1, 2, 3, 3, 6, 5], dtype=torch.int32).repeat(B, 1).cuda()
    kept = [torch.zeros((2, 0, H, D), dtype=torch.bfloat16) for _ in range(B)]
    head = torch.randn((H * G * D, V), generator=g).cuda() * 0.2
    for _ in range(3):
        rows = _bf(g, 2, B, T, H, D).cuda()
        q = _bf(g, B, T, H * G, D).cuda()
        ks, vs = (None, None) if scale is None else (scale[0], scale[1])
        out = sv.verify_attention(q, cache[0], cache[1], lens, k_new=rows[0], v_new=rows[1], parent=parent,
                                  k_scale=ks, v_scale=vs)
        kk = torch.zeros((B, L, H, D), dtype=torch.bfloat16)
        vv = torch.zeros((B, L, H, D), dtype=torch.bfloat16)
        for b in range(B):
            kk[b, :kept[b].shape[1]], vv[b, :kept[b].shape[1]] = kept[b][0], kept[b][1]
        sk = sw = None
        if dt == FP8:
            kk, sk = ref.quantise(kk)
            vv, sw = ref.quantise(vv)
        o, _, tol, _ = ref.attention(q.cpu(), kk, vv, lens.tolist(), rows[0].cpu(), rows[1].cpu(), parent.cpu(), ks=sk, vs=sw)
        ref.assert_close(out, o, tol, "out")
        logits = out.float().reshape(B, T, -1) @ head
        tokens = torch.randint(0, V, (B, T), generator=g, dtype=torch.int32).cuda()
        tokens[:, 1] = logits[:, 0].argmax(-1)               # the root's first child is accepted
        tokens[:2, 3] = logits[:2, 1].argmax(-1)
        _, path, acc = ctx.tree_run(logits, None, parent, tokens, None, None, greedy=True)
        sv.kv_commit_path(rows, cache, lens, acc, path=path, lead=1, scale=scale)
        for b in range(B):
            src = [0] + path[b, :int(acc[b])].tolist()
            kept[b] = torch.cat([kept[b], rows[:, b, src].cpu()], 1)
        assert lens.tolist() == [x.shape[1] for x in kept]
        assert all(int(acc[b]) >= 1 for b in range(B))
    if dt == FP8:
        back = sv.kv_read(cache, scale, lens).cpu()
        for b in range(B):
            n = kept[b].shape[1]
            codes, s = ref.quantise(kept[b])
            assert torch.equal(back[:, b, :n].double(), ref.values(codes, s))
            assert (back[:, b, n:] == 0).all()
    assert ctx.status() == sv.SV_OK
    ctx.close()
