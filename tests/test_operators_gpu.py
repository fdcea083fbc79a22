"""Tree attention, read-back and rotary positions on the GPU, against plain 64-bit
computations over the oracle's dequantised tokens."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from harness import Pair

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def K():
    import quantised_kv_cache_kvq_gb300 as K
    return K


# ------------------------------------------------------------------------------ caches
def wrap(K, pair):
    """The pair's GPU cache behind the binding's class."""
    c = K.QuantizedKVCache.__new__(K.QuantizedKVCache)
    c.cfg, c.device, c.cache, c.workspace = pair.lib_cfg, torch.device("cuda", 0), pair.gpu, pair.ws
    c.nbytes, c._tree_workspaces = pair.nbytes, {}
    return c


def filled(lengths, seed=0, scale=1.0, layers=1, layer=0, **kw):
    """A pair of caches whose sequences hold `lengths` tokens."""
    gen = torch.Generator().manual_seed(seed)
    p = Pair(batch=len(lengths), layers=layers, **kw)
    k, v = p.rand_kv(len(lengths), max(lengths), gen, scale=scale)
    sc = None
    if p.kw["scheme"] in (2, 3):
        top = 448.0 if p.kw["scheme"] == 2 else 57344.0
        sc = torch.stack([x.float().abs().amax(dim=(0, 1, 3)) / top for x in (k, v)], 1) + 1e-6
    if max(lengths):
        p.append(layer, k, v, n_valid=list(lengths), fp8_scales=sc)
    return p, gen


def tokens64(p, layer=0):
    """[batch] lists of (keys, values) [tokens][kv_heads][head_dim] float64 as the oracle
    dequantises them."""
    got = []
    H, D = p.kw["kv_heads"], p.kw["head_dim"]
    for b in range(p.kw["batch"]):
        n, _ = p.img.state(layer, b)
        k, v = np.zeros((n, H, D), np.float32), np.zeros((n, H, D), np.float32)
        for h in range(H):
            for t in range(n):
                k[t, h], v[t, h] = p.img.dequant_token(layer, b, h, t)
        got.append((k, v))
    return got


def shuffled_table(lengths, residual, group_k, page_groups, max_tokens, seed=5):
    ng = max(0, max_tokens - residual) // group_k
    mp = -(-ng // page_groups)
    rng = np.random.RandomState(seed)
    pool = len(lengths) * mp + 3
    return pool, rng.permutation(pool)[:len(lengths) * mp].reshape(len(lengths), mp).astype(np.int32)


CACHES = [
    dict(bits=2, lengths=(300, 1, 0, 97), max_tokens=320),
    dict(bits=4, group_k=128, group_v=128, residual=16, lengths=(513, 144), max_tokens=600),
    dict(bits=8, group_k=48, group_v=64, head_dim=64, residual=20, lengths=(333, 70), max_tokens=400, q_heads=2),
    dict(bits=2, group_k=16, group_v=16, head_dim=256, residual=0, lengths=(200, 16, 15), max_tokens=256, q_heads=16),
    dict(bits=4, group_k=80, group_v=32, residual=1, lengths=(400, 81), max_tokens=401, kv_heads=3, q_heads=12),
    dict(bits=2, group_k=32, group_v=64, outliers=2, lengths=(290, 161), max_tokens=300, paged=3),
    dict(bits=8, group_k=16, group_v=16, head_dim=128, outliers=4, lengths=(150,), max_tokens=160, residual=5),
    dict(bits=4, group_k=64, group_v=32, rope_base=10000.0, lengths=(280, 65), max_tokens=300),
    dict(bits=2, group_k=32, group_v=32, rope_base=500000.0, outliers=1, lengths=(270, 3), max_tokens=300, paged=1),
    dict(bits=2, group_k=16, group_v=16, head_dim=256, outliers=3, lengths=(150, 40), max_tokens=160, residual=5, q_heads=4, paged=2),
    dict(bits=4, group_k=16, group_v=16, head_dim=256, outliers=2, lengths=(100,), max_tokens=160, residual=0, rope_base=10000.0,
         q_heads=8),
    dict(scheme="int8", head_dim=32, lengths=(257, 128, 0), max_tokens=300),
    dict(scheme="int8", head_dim=256, lengths=(129, 16), max_tokens=130, q_heads=2),
    dict(scheme="int4", head_dim=64, lengths=(300, 2), max_tokens=301),
    dict(scheme="int4", head_dim=32, lengths=(40, 1), max_tokens=64, q_heads=16),
    dict(scheme="fp8", head_dim=128, lengths=(311, 0, 17), max_tokens=320, q_heads=16),
    dict(scheme="fp8e5m2", head_dim=32, lengths=(100, 255), max_tokens=256),
    dict(scheme="fp8", head_dim=256, lengths=(64, 131), max_tokens=131, kv_heads=1, q_heads=4),
]


def make(case, **more):
    kw = dict(case, **more)
    lengths, paged = kw.pop("lengths"), kw.pop("paged", 0)
    if paged:
        pool, table = shuffled_table(lengths, kw.get("residual", 32), kw["group_k"], paged, kw["max_tokens"])
        kw.update(page_groups=paged, num_pages=pool, block_table=table)
    return filled(lengths, **kw)


# ------------------------------------------------------------------------------ read-back
@pytest.mark.parametrize("case", CACHES, ids=str)
def test_read_is_the_oracles_dequantised_value(K, case):
    p, _ = make(case)
    cache = wrap(K, p)
    B, n = p.kw["batch"], max(case["lengths"])
    want = [np.zeros((B, n + 3, p.kw["kv_heads"], p.kw["head_dim"]), np.float32) for _ in range(2)]
    for b, kv in enumerate(tokens64(p)):
        for w, x in zip(want, kv):
            w[b, :x.shape[0]] = x
    for first, count in ((0, n + 3), (0, 1), (n // 2, n - n // 2), (n - 1, 3), (17, 30)):
        for dtype in ("f32", "bf16"):
            got = cache.read(0, first=first, count=count, dtype=dtype)
            for g, w in zip(got, want):
                ref = torch.zeros(B, count, *w.shape[2:])
                have = torch.from_numpy(w[:, first:first + count])
                ref[:, :have.shape[1]] = have
                assert torch.equal(g.cpu(), ref.to(g.dtype)), (first, count, dtype)
    assert p.status() == 0


def test_read_from_each_sequences_own_start(K):
    p, _ = make(dict(bits=2, lengths=(300, 150, 40, 0), max_tokens=320))
    cache = wrap(K, p)
    starts = [290, -7, 38, 5]
    whole = cache.read(0, count=320, dtype="f32")
    got = cache.read(0, first=torch.tensor(starts[1:], dtype=torch.int32, device="cuda"), seq_begin=1, count=20,
                     dtype="f32")
    for g, w in zip(got, whole):
        for i, b in enumerate((1, 2, 3)):
            for j in range(20):
                t = starts[b] + j
                assert torch.equal(g[i, j], w[b, t] if t >= 0 else torch.zeros_like(w[b, 0]))


def test_read_one_of_keys_and_values_and_into_given_tensors(K):
    p, _ = make(dict(bits=4, lengths=(100, 90), max_tokens=128))
    k, v = wrap(K, p).read(0, count=100)
    k2 = torch.full_like(k, 7.0)
    K.kvq_read_tokens(p.lib_cfg, p.gpu, 0, 0, 2, None, 0, 100, k2, None)
    v2 = torch.full_like(v, 7.0)
    K.kvq_read_tokens(p.lib_cfg, p.gpu, 0, 0, 2, None, 0, 100, None, v2)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    before = torch.full((4, 100, 2, 128), 3.0, dtype=BF16, device="cuda")     # rows before and behind stay
    out = before.clone()
    wrap(K, p).read(0, count=100, k_out=out[1:3], v_out=torch.empty_like(v))
    assert torch.equal(out[0], before[0]) and torch.equal(out[3], before[3]) and torch.equal(out[1:3], k)


@pytest.mark.parametrize("case", [
    dict(bits=2, group_k=16, group_v=16, head_dim=64), dict(bits=4, group_k=48, group_v=32, outliers=2, head_dim=128),
    dict(bits=8, group_k=32, group_v=64, head_dim=256), dict(scheme="int8", head_dim=32), dict(scheme="int4", head_dim=128),
    dict(scheme="fp8", head_dim=64), dict(scheme="fp8e5m2", head_dim=256)], ids=str)
def test_read_of_many_tiles_is_the_read_of_its_pieces(K, case):
    """Large reads run other blocks than small ones (test_read_is_the_oracles_dequantised_value)."""
    scheme = case.get("scheme", "kivi")
    B, H, n, D = 3, 12, 4000, case["head_dim"]
    kw = {x: case[x] for x in ("bits", "group_k", "group_v", "outliers") if x in case}
    cache = K.QuantizedKVCache(K.make_config(scheme, 1, B, H, H, D, n, residual=37 if scheme == "kivi" else 0, **kw))
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(B, n, H, D, generator=gen, device="cuda").to(BF16) for _ in range(2))
    scales = torch.full((H, 2), 0.01, device="cuda")
    counts = torch.tensor([n, n - 133, 17], dtype=torch.int32, device="cuda")
    cache.append(0, k, v, n_valid=counts, fp8_scales=scales)
    for dtype in ("bf16", "f32"):
        whole = cache.read(0, count=n, dtype=dtype)
        for b, first in ((0, 0), (0, n - 100), (1, n - 200), (2, 0), (1, 1111)):
            piece = cache.read(0, first=first, count=100, seq_begin=b, seq_count=1, dtype=dtype)
            for w, x in zip(whole, piece):
                assert torch.equal(w[b, first:first + 100], x[0])


def test_read_reports_a_page_outside_the_pool(K):
    case = dict(bits=2, group_k=32, group_v=32, lengths=(300, 300), max_tokens=320, paged=2)
    p, _ = make(case)
    good = wrap(K, p).read(0, count=300)
    table = p.lib_cfg._table.cpu().numpy().copy()
    table[1, 0] = 10 ** 6
    p.lib_cfg.set_block_table(torch.from_numpy(table).cuda())
    bad = wrap(K, p).read(0, count=300)
    assert p.status() == K.KVQ_STATUS_BAD_PAGE
    for g, x in zip(good, bad):
        assert torch.equal(g[0], x[0]) and torch.equal(g[1, 64:], x[1, 64:]) and not x[1, :64].any()


# ------------------------------------------------------------------------------ tree attention
def tree64(p, layer, q, dk, dv, mask, nodes, scale):
    """(outputs, error bounds) [batch][nodes][q_heads][head_dim] in 64 bits.  The bound, per
    element: keys are rounded to binary16 (relative 2^-11; twice where the rotation follows
    the dequantisation, whose binary32 sine is 1e-6 off), so a score s = scale q.k is off by
    at most d = |scale| sum |q k| (2^-11 or 2 * 2^-11 + 2e-6) + 2^-20 |s| (binary32), a weight
    by a factor e^(2 d), and weights and values are rounded once (2^-11 each): the output is
    off by (e^(2 d) - 1 + 2 * 2^-11 + 2^-18) sum p |v|, and its bf16 rounding by 2^-8 of it.
    Under the kernels' power-of-two scales a value under 2^-28 of the largest of its tile
    is rounded to a step of 2^-39 of that: 1e-6 of the largest value is room for it."""
    B, T, Hq, D = q.shape
    g = Hq // p.kw["kv_heads"]
    out, tol = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq, D))
    rope = p.kw["rope_base"]
    rel = 2 * 2.0 ** -11 + 2e-6 if rope else 2.0 ** -11
    q, dk, dv = (x.float().cpu().numpy().astype(np.float64) for x in (q, dk, dv))
    for b, (k, v) in enumerate(tokens64(p, layer)):
        t = T if nodes is None else nodes[b]
        for h in range(p.kw["kv_heads"]):
            kk = k[:, h].astype(np.float64)
            if rope:
                kk = np.array([O.rope_key(k[i, h], i, rope) for i in range(len(k))]).reshape(-1, D)
            kk, vv = np.concatenate([kk, dk[b, :t, h]]), np.concatenate([v[:, h].astype(np.float64), dv[b, :t, h]])
            for i in range(t):
                see = np.ones(len(kk), bool)
                see[len(k):] = (np.arange(t) <= i) if mask is None else mask[b, i, :t]
                if not see.any():
                    continue
                ks, vs = kk[see], vv[see]
                for x in range(h * g, (h + 1) * g):
                    s = ks @ q[b, i, x] * scale
                    d = (abs(scale) * (np.abs(ks) @ np.abs(q[b, i, x])) * rel + 2.0 ** -20 * np.abs(s)).max()
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[b, i, x] = w @ vs
                    tol[b, i, x] = (np.expm1(2 * d) + 2.0 ** -10 + 2.0 ** -18) * (w @ np.abs(vs)) \
                        + 2.0 ** -8 * np.abs(out[b, i, x]) + 1e-6 * np.abs(vs).max()
    return out, tol


def drafts(p, nodes, gen, tree=True):
    B, Hq, H, D = (p.kw[x] for x in ("batch", "q_heads", "kv_heads", "head_dim"))
    q = torch.randn(B, nodes, Hq, D, generator=gen).to(BF16)
    dk = torch.randn(B, nodes, H, D, generator=gen).to(BF16)
    dv = torch.randn(B, nodes, H, D, generator=gen).to(BF16)
    mask = None
    if tree:
        mask = torch.zeros(B, nodes, nodes, dtype=torch.bool)
        for b in range(B):
            for i in range(nodes):
                if i:
                    mask[b, i] = mask[b, int(torch.randint(0, i, (1,), generator=gen))]
                mask[b, i, i] = True
    return q, dk, dv, mask


def check_tree(K, p, q, dk, dv, mask, nodes=None, layer=0, scale=None, rows=None):
    cache = wrap(K, p)
    scale = 1.0 / math.sqrt(p.kw["head_dim"]) if scale is None else scale
    nn = None if nodes is None else torch.tensor(nodes, dtype=torch.int32, device="cuda")
    got = cache.tree_decode(layer, q.cuda(), dk.cuda(), dv.cuda(), None if mask is None else mask.cuda(), nn, scale)
    ref, tol = tree64(p, layer, q, dk, dv, None if mask is None else mask.numpy(), nodes, scale)
    got = got.float().cpu().numpy().astype(np.float64)
    err = np.abs(got - ref)
    ok = err <= tol
    if rows is not None:
        ok = ok[rows]
    assert ok.all(), "%d of %d outside, worst %r" % ((~ok).sum(), ok.size, np.unravel_index(np.nanargmax(err - tol), err.shape))
    assert cache.status() == 0
    return got


@pytest.mark.parametrize("nodes", [1, 5, 17])
@pytest.mark.parametrize("case", CACHES, ids=str)
def test_tree_over_every_cache(K, case, nodes):
    p, gen = make(case)
    check_tree(K, p, *drafts(p, nodes, gen))


@pytest.mark.parametrize("nodes", [2, 3, 8, 16, 31, 64, 65, 130, 256])
@pytest.mark.parametrize("gqa", [1, 8])
def test_tree_sizes(K, nodes, gqa):
    p, gen = make(dict(bits=2, lengths=(200, 37), max_tokens=208, kv_heads=1, q_heads=gqa))
    check_tree(K, p, *drafts(p, nodes, gen))


def test_tree_chain_equals_its_mask(K):
    p, gen = make(dict(bits=4, lengths=(260, 130), max_tokens=300))
    q, dk, dv, _ = drafts(p, 21, gen, tree=False)
    a = check_tree(K, p, q, dk, dv, None)
    b = check_tree(K, p, q, dk, dv, torch.ones(2, 21, 21).tril().bool())
    assert np.array_equal(a, b)


def test_tree_of_one_draft_is_the_decode_after_its_append(K):
    p, gen = make(dict(bits=2, lengths=(300, 64), max_tokens=320))
    q, dk, dv, _ = drafts(p, 1, gen, tree=False)
    tree = check_tree(K, p, q, dk, dv, None)[:, 0]
    ref, tol = (x[:, 0] for x in tree64(p, 0, q, dk, dv, None, None, 1.0 / math.sqrt(128)))
    p.append(0, dk, dv)
    out = torch.empty(q.shape[0], *q.shape[2:], device="cuda")
    K.kvq_decode_attention(p.lib_cfg, p.gpu, 0, q[:, 0].contiguous().cuda(), 1.0 / math.sqrt(128), out, p.ws)
    # the append leaves the draft in the window (no group completes), so both compute the same
    # attention: the tree is within its bound of the 64-bit value (check_tree), the decode within
    # its own tolerance, and so the two within their sum of each other
    assert [p.img.state(0, b)[1] for b in range(2)] == [256, 32]
    assert (np.abs(tree - out.cpu().numpy()) <= tol + 2e-3 + 1e-2 * np.abs(ref)).all()


def test_tree_masks_padding_and_empty_rows(K):
    p, gen = make(dict(bits=2, lengths=(150, 0, 0, 77), max_tokens=160))
    q, dk, dv, mask = drafts(p, 12, gen)
    mask[1, 4] = False          # no cached token and no visible draft: 0
    mask[3, 2] = False          # the cached tokens alone
    mask[0, 3, 11] = True       # a later node
    got = check_tree(K, p, q, dk, dv, mask, nodes=[12, 7, 0, 5])
    assert not got[1, 4].any() and not got[1, 7:].any() and not got[2].any() and not got[3, 5:].any()
    assert got[1, 3].any()


def test_tree_leaves_no_trace_of_masked_or_padding_drafts(K):
    p, gen = make(dict(bits=4, lengths=(140, 20), max_tokens=160))
    q, dk, dv, mask = drafts(p, 20, gen)
    mask[:, :, 9] = False
    nodes = [15, 20]
    clean = check_tree(K, p, q, dk, dv, mask, nodes)
    for bad in (math.nan, math.inf, -math.inf, 3.0e38, torch.finfo(BF16).min):
        k2, v2, q2 = dk.clone(), dv.clone(), q.clone()
        k2[:, 9], v2[:, 9] = bad, bad                    # seen by nobody
        k2[0, 15:], v2[0, 15:], q2[0, 15:] = bad, bad, bad   # padding
        got = check_tree(K, p, q2, k2, v2, mask, nodes)
        assert np.array_equal(got, clean), bad


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_tree_nonfinite_draft_values_reach_only_the_rows_that_see_them(K, bad):
    p, gen = make(dict(bits=2, lengths=(100, 10), max_tokens=160))
    q, dk, dv, mask = drafts(p, 10, gen)
    mask = torch.eye(10, dtype=torch.bool).expand(2, 10, 10).clone()
    mask[0, 7, 4] = True
    clean = check_tree(K, p, q, dk, dv, mask)
    v2 = dv.clone()
    v2[:, 4, 1, 5] = bad
    cache = wrap(K, p)
    got = cache.tree_decode(0, q.cuda(), dk.cuda(), v2.cuda(), mask.cuda()).float().cpu().numpy()
    hit = np.zeros(got.shape, bool)
    hit[0, 7, 4:, 5] = hit[:, 4, 4:, 5] = True          # query heads 4..7 read KV head 1
    assert np.array_equal(got[~hit], clean[~hit].astype(np.float32))
    assert (np.isnan(got[hit]) if math.isnan(bad) else got[hit] == bad).all()


@pytest.mark.parametrize("kscale,vscale", [(1e30, 1.0), (1.0, 1e30), (1e-30, 1e-30), (1e4, 1e6)])
@pytest.mark.parametrize("scheme", ["kivi", "int8", "fp8"])
def test_tree_holds_the_types_range(K, scheme, kscale, vscale):
    """Values far outside binary16's range: KIVI's own binary16 parameters stay within it, its
    window and the drafts do not."""
    gen = torch.Generator().manual_seed(3)
    p = Pair(scheme=scheme, batch=1, q_heads=4, kv_heads=1, max_tokens=200)
    big = scheme != "kivi"
    for part, (ks, vs) in enumerate(((kscale, vscale) if big else (1.0, 1.0), (kscale, vscale))):
        n = 130 if part == 0 else 20
        k, v = p.rand_kv(1, n, gen)
        sc = None
        if scheme == "fp8":
            sc = torch.tensor([[kscale * 0.2, vscale * 0.2]])
        p.append(0, (k.float() * ks).to(BF16), (v.float() * vs).to(BF16), fp8_scales=sc)
    q, dk, dv, mask = drafts(p, 6, gen)
    check_tree(K, p, q, (dk.float() * kscale).to(BF16), (dv.float() * vscale).to(BF16), mask,
               scale=0.1 / kscale if kscale > 1 else 0.1)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_tree_scales(K, scale):
    p, gen = make(dict(bits=2, lengths=(300,), max_tokens=320, scale=0.3))
    check_tree(K, p, *drafts(p, 9, gen), scale=scale)


def test_tree_growing_scores(K):
    """Keys that grow along the context, so that the running maximum moves in every tile."""
    gen = torch.Generator().manual_seed(8)
    p = Pair(bits=4, batch=1, q_heads=4, kv_heads=1, group_k=32, group_v=32, max_tokens=900)
    k, v = p.rand_kv(1, 900, gen, outliers=False)
    k = (k.float() * torch.linspace(0.05, 3.0, 900).view(1, -1, 1, 1)).to(BF16)
    p.append(0, k, v)
    check_tree(K, p, *drafts(p, 7, gen))
    p2 = Pair(bits=4, batch=1, q_heads=4, kv_heads=1, group_k=32, group_v=32, max_tokens=900)
    p2.append(0, k.flip(1).contiguous(), v)
    check_tree(K, p2, *drafts(p2, 7, gen))


def test_tree_of_a_later_layer_and_over_the_unflushed_window(K):
    p, gen = filled((120, 50), layers=3, layer=2, max_tokens=300)
    k, v = p.rand_kv(2, 8, gen)           # the windows, of 64 tokens, hold 64 and 58
    p.append(2, k, v, flags=K.KVQ_NO_AUTOFLUSH)
    check_tree(K, p, *drafts(p, 6, gen), layer=2)


def test_tree_split_contexts(K):
    """One long context over many blocks beside empty and short ones."""
    p, gen = make(dict(bits=2, lengths=(6000, 0, 33), max_tokens=6016, kv_heads=1, q_heads=4))
    check_tree(K, p, *drafts(p, 5, gen), nodes=[5, 5, 0])


@pytest.mark.parametrize("gqa,nodes", [(1, 3), (8, 40)])
def test_tree_of_more_sequences_than_threads(K, gqa, nodes):
    gen = torch.Generator().manual_seed(4)
    lengths = torch.randint(0, 40, (600,), generator=gen).tolist()
    p, gen = make(dict(bits=2, head_dim=64, kv_heads=1, q_heads=gqa, lengths=lengths, max_tokens=64, residual=8))
    counts = torch.randint(-1, nodes + 3, (600,), generator=gen).tolist()      # out of range: as the nearest in it
    q, dk, dv, mask = drafts(p, nodes, gen)
    cache = wrap(K, p)
    got = cache.tree_decode(0, q.cuda(), dk.cuda(), dv.cuda(), mask.cuda(),
                            torch.tensor(counts, dtype=torch.int32, device="cuda")).float().cpu().numpy()
    some = [0, 255, 256, 257, 511, 512, 598, 599] + list(range(100, 130))
    few = [min(max(c, 0), nodes) if b in some else 0 for b, c in enumerate(counts)]
    ref, tol = tree64(p, 0, q, dk, dv, mask.numpy(), few, 0.125)
    assert (np.abs(got - ref) <= tol)[some].all()
    for b, c in enumerate(counts):
        assert not got[b, max(c, 0):].any()


@pytest.mark.parametrize("case", [dict(scheme="int8", head_dim=64), dict(scheme="int4", head_dim=32), dict(scheme="fp8", head_dim=128),
                                  dict(bits=2, head_dim=64, group_k=16, group_v=16, residual=20, paged=3)], ids=str)
def test_tree_of_many_short_sequences(K, case):
    """Several sequences to a block, some empty or without drafts: its copies run ahead from one to
    the next."""
    gen = torch.Generator().manual_seed(8)
    lengths = torch.randint(0, 300, (200,), generator=gen).tolist()
    lengths[7:12] = [0, 0, 299, 0, 128]
    p, gen = make(dict(case, kv_heads=4, q_heads=8, lengths=lengths, max_tokens=300))
    counts = torch.randint(0, 4, (200,), generator=gen).tolist()
    q, dk, dv, mask = drafts(p, 3, gen)
    cache = wrap(K, p)
    got = cache.tree_decode(0, q.cuda(), dk.cuda(), dv.cuda(), mask.cuda(),
                            torch.tensor(counts, dtype=torch.int32, device="cuda")).float().cpu().numpy()
    ref, tol = tree64(p, 0, q, dk, dv, mask.numpy(), counts, 1.0 / math.sqrt(p.kw["head_dim"]))
    assert (np.abs(got - ref) <= tol).all() and cache.status() == 0


def test_tree_replayed_over_a_growing_cache(K):
    p, gen = make(dict(bits=4, lengths=(250, 60), max_tokens=900))
    cache = wrap(K, p)
    q, dk, dv, mask = drafts(p, 6, gen)
    args = [x.cuda() for x in (q, dk, dv, mask)]
    ws, out = cache.tree_workspace(6), torch.zeros(q.shape, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.tree_decode(0, *args, out=out, workspace=ws)
    for n in (1, 300, 17):
        p.append(0, *p.rand_kv(2, n, gen))
        g.replay()
        torch.cuda.synchronize()
        ref, tol = tree64(p, 0, q, dk, dv, mask.numpy(), None, 1.0 / math.sqrt(128))
        assert (np.abs(out.float().cpu().numpy() - ref) <= tol).all()


def test_tree_queries_of_very_different_sizes(K):
    """A query far larger than the others, or not finite, changes nothing for them."""
    p, gen = make(dict(bits=2, lengths=(200, 64), max_tokens=208))
    q, dk, dv, mask = drafts(p, 9, gen)
    clean = check_tree(K, p, q, dk, dv, mask)
    for big in (1e30, math.inf, math.nan):
        q2 = q.clone()
        q2[:, 4] *= big
        got = wrap(K, p).tree_decode(0, q2.cuda(), dk.cuda(), dv.cuda(), mask.cuda()).float().cpu().numpy()
        ref, tol = tree64(p, 0, q, dk, dv, mask.numpy(), None, 1.0 / math.sqrt(128))
        others = [i for i in range(9) if i != 4]
        assert (np.abs(got - ref) <= tol)[:, others].all()
    assert np.isfinite(clean).all()


def test_tree_is_repeatable_and_captured(K):
    """Twice the same bits; a captured step replays on new inputs; two graphs with workspaces of
    their own, replayed side by side on two streams."""
    p, gen = make(dict(bits=2, lengths=(2000, 700), max_tokens=2048))
    cache = wrap(K, p)
    q, dk, dv, mask = (x.cuda() for x in drafts(p, 13, gen))
    q2 = torch.randn(q.shape, generator=gen).to(BF16).cuda()
    a, b, a2 = (cache.tree_decode(0, x, dk, dv, mask) for x in (q, q, q2))
    assert torch.equal(a, b)
    graphs = []
    for x in (q, q2):
        ws, xin, out = cache.tree_workspace(13), x.clone(), torch.zeros_like(a)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.tree_decode(0, xin, dk, dv, mask, out=out, workspace=ws)
        graphs.append((g, xin, out, torch.cuda.Stream(), ws))
    for _ in range(3):
        for g, _, out, s, _ in graphs:
            out.zero_()
        torch.cuda.synchronize()
        for g, _, _, s, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][2], a) and torch.equal(graphs[1][2], a2)
    graphs[0][1].copy_(q2)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][2], a2)


def test_tree_captured_before_its_workspace_is_made_is_refused(K):
    """A workspace that the cache keeps is not made of a graph's memory."""
    p, gen = make(dict(bits=2, lengths=(200, 100), max_tokens=208))
    cache = wrap(K, p)
    q, dk, dv, mask = (x.cuda() for x in drafts(p, 5, gen))
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out.fill_(1.0)
        with pytest.raises(ValueError, match="before the capture"):
            cache.tree_decode(0, q, dk, dv, mask, out=out)
    want = cache.tree_decode(0, q, dk, dv, mask)            # makes it
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.tree_decode(0, q, dk, dv, mask, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and cache.status() == 0


def test_tree_from_page_locked_host_memory_on_another_stream(K):
    p, gen = make(dict(bits=2, lengths=(200, 100), max_tokens=208))
    cache = wrap(K, p)
    q, dk, dv, mask = drafts(p, 7, gen)
    want = cache.tree_decode(0, q.cuda(), dk.cuda(), dv.cuda(), mask.cuda())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    pinned = [x.pin_memory() for x in (q, dk, dv, mask)]
    out = torch.zeros(q.shape, dtype=BF16).pin_memory()
    cache.tree_decode(0, *pinned, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want.cpu())


def test_tree_reports_a_page_outside_the_pool(K):
    case = dict(bits=2, group_k=32, group_v=32, lengths=(300, 300), max_tokens=320, paged=2)
    p, gen = make(case)
    q, dk, dv, mask = drafts(p, 4, gen)
    good = check_tree(K, p, q, dk, dv, mask)
    table = p.lib_cfg._table.cpu().numpy().copy()
    table[1, 1] = -1
    p.lib_cfg.set_block_table(torch.from_numpy(table).cuda())
    cache = wrap(K, p)
    got = cache.tree_decode(0, q.cuda(), dk.cuda(), dv.cuda(), mask.cuda()).float().cpu().numpy()
    assert cache.status() == K.KVQ_STATUS_BAD_PAGE
    assert np.array_equal(got[0], good[0].astype(np.float32))


@pytest.mark.parametrize("op", ["decode", "tree"])
def test_layouts_that_share_a_kernel_take_turns(K, op):
    """A layout with more shared memory than the one that ran in between launches again."""
    pairs = [make(dict(bits=4, group_k=g, group_v=128, lengths=(300,), max_tokens=320, residual=16)) for g in (128, 80)]
    for p, gen in pairs + pairs:
        if op == "decode":
            got, ref = p.decode(0, p.rand_q(gen))
            assert (np.abs(got - ref) <= 2e-3 + 1e-2 * np.abs(ref)).all()
        else:
            check_tree(K, p, *drafts(p, 3, gen))


# ------------------------------------------------------------------------------ rotary positions
def rope64(x, pos, w, R, layout, magnitude, transpose):
    """(result, error bound) of rotating x [tokens][heads][D]: the angle is the binary32
    product; sine and cosine are 2^-22 off in binary32, times the magnitude and in two
    products and a sum 2^-23 more; then the rounding to the type."""
    y = x.double().cpu().numpy()
    angle = (pos.cpu().float()[:, None] * torch.tensor(w)[None]).double().numpy()[:, None]
    c, s = np.cos(angle) * magnitude, np.sin(angle) * magnitude * (-1 if transpose else 1)
    i = np.arange(R // 2)
    a, b = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
    out, tol = y.copy(), np.zeros_like(y)
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    tol[..., a] = tol[..., b] = (np.abs(y[..., a]) + np.abs(y[..., b])) * abs(magnitude) * 3 * 2.0 ** -23
    # copied channels are exact
    return out, tol + np.where(tol > 0, torch.finfo(x.dtype).eps / 2 * np.abs(out), 0.0)


@pytest.mark.parametrize("dtype", [BF16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,Hq,H,D,R", [(1, 1, 1, 2, 2), (7, 32, 8, 128, 128), (33, 3, 1, 96, 48), (5, 8, 8, 64, 2),
                                             (3, 1, 2, 80, 20), (700, 2, 1, 256, 256), (4, 5, 1, 1024, 256),
                                             (9, 4, 2, 7, 6)])
def test_rope(K, dtype, layout, tokens, Hq, H, D, R):
    gen = torch.Generator().manual_seed(tokens)
    r = K.RotaryEmbedding(D, 500000.0, rotary_dim=R, layout=layout, magnitude=1.25)
    w = list(r.frequencies)
    rows = torch.randn(tokens, Hq + 2 * H, D, generator=gen).to(dtype).cuda()
    q, k = rows[:, :Hq], rows[:, Hq:Hq + H]
    for top in (64, 200000, 2 ** 31 - 1):
        pos = torch.randint(0, top, (tokens,), generator=gen, dtype=torch.int32).cuda()
        pos[0] = top - 1
        for transpose in (False, True):
            got = r.rotate(q, k, pos, transpose=transpose)
            for x, y in zip((q, k), got):
                ref, tol = rope64(x, pos, w, R, layout, 1.25, transpose)
                assert y.dtype == dtype and (np.abs(y.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("offset,extra", [(0, 0), (1, 1), (2, 6), (4, 4), (8, 8)])
def test_rope_alignments_strides_and_in_place(K, offset, extra):
    gen = torch.Generator().manual_seed(1)
    T, H, D = 11, 4, 64
    flat = torch.randn(T * (H * D + extra) + offset + 16, generator=gen).to(BF16).cuda()
    x = flat[offset:].as_strided((T, H, D), (H * D + extra, D, 1))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1000
    r = K.RotaryEmbedding(D, rotary_dim=32)
    want, _ = r.rotate(x.contiguous(), None, pos)
    assert r.rotate(None, x, pos)[0] is None
    assert torch.equal(r.rotate(None, x, pos)[1], want)
    before = flat.clone()
    got, _ = r.rotate(x, None, pos, q_out=x)                      # in place
    assert got.data_ptr() == x.data_ptr() and torch.equal(x, want)
    y = before[offset:].as_strided((T, H, D), (H * D + extra, D, 1))
    y.copy_(want)
    assert torch.equal(flat, before)                              # nothing between the rows was written


def test_rope_gradient(K):
    """The transposed product is the gradient: <R x, y> = <x, R^T y>, and differences of R."""
    gen = torch.Generator().manual_seed(2)
    for layout in ("half", "interleaved"):
        r = K.RotaryEmbedding(64, rotary_dim=48, layout=layout, magnitude=1.1, scaling="by_parts", factor=8.0)
        x, y = (torch.randn(20, 3, 64, generator=gen).cuda() for _ in range(2))
        pos = torch.randint(0, 9000, (20,), generator=gen, dtype=torch.int32).cuda()
        rx, _ = r.rotate(x, None, pos)
        ry, _ = r.rotate(y, None, pos, transpose=True)
        a, b = (rx.double() * y.double()).sum(), (x.double() * ry.double()).sum()
        # each element is 3 * 2^-23 (|a| + |b|) m off: summed over the products' magnitudes
        room = 8 * 2.0 ** -23 * 1.1 * (x.abs().double().sum() * y.abs().max()).item()
        assert abs(a - b).item() <= room
        d = torch.zeros_like(x)
        d[4, 1, 10] = 0.5
        step = (r.rotate(x + d, None, pos)[0] - rx).double() / 0.5
        col = torch.zeros_like(x)
        for j in range(64):                                       # column 10 of R against rows of R^T
            e = torch.zeros_like(x)
            e[4, 1, j] = 1.0
            col[4, 1, j] = r.rotate(e, None, pos, transpose=True)[0][4, 1, 10]
        # x + d and the two results are rounded to binary32 under 8: 2^-22 each, over 0.5
        assert (step - col.double()).abs().max().item() <= 4 * 2.0 ** -22 / 0.5 * 4


def test_rope_captured(K):
    r = K.RotaryEmbedding(128, 500000.0)
    x = torch.randn(6, 4, 128, device="cuda").to(BF16)
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.rotate(x, None, pos, q_out=out)
    pos.add_(100)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, r.rotate(x, None, pos)[0])


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("rope_base", [0.0, 10000.0])
def test_a_verification_step(K, rope_base):
    """Rotate the drafts, attend through the tree, append the accepted path, read it back; the
    next step's root sees what a decode of the same query sees."""
    B, T, Hq, H, D = 2, 9, 8, 2, 128
    p, gen = make(dict(bits=4, lengths=(200, 90), max_tokens=260, rope_base=rope_base))
    cache, r = wrap(K, p), K.RotaryEmbedding(D, 10000.0)
    n, _ = cache.lengths(0)
    q, dk, dv, mask = drafts(p, T, gen)
    depth = mask.sum(2).int().cuda() - 1
    pos = (n.view(B, 1) + depth).reshape(-1)
    rows = torch.cat([q, dk, dv], 2).cuda().view(B * T, Hq + 2 * H, D)       # a fused projection
    qr, kr = r.rotate(rows[:, :Hq], rows[:, Hq:Hq + H], pos)
    qr, kr = qr.view(B, T, Hq, D), kr.view(B, T, H, D)
    check_tree(K, p, qr.cpu(), kr.cpu(), dv, mask)
    path = [i for i in range(T) if mask[0, T - 1, i]]                       # the last node's ancestors
    assert path[-1] == T - 1
    take = torch.tensor(path)
    ks = (dk if rope_base else kr.cpu())[:, take].contiguous()             # pre-RoPE caches take keys as given
    p.append(0, ks, dv[:, take].contiguous(), n_valid=[len(path), 1])
    after, _ = cache.lengths(0)
    assert after.tolist() == [200 + len(path), 91]
    k, v = cache.read(0, first=n, count=len(path))
    if p.img.state(0, 0)[1] <= 200:                                          # still in the bf16 window
        assert torch.equal(k[0].cpu(), ks[0]) and torch.equal(v[0].cpu(), dv[0, take])
    q2, dk2, dv2, mask2 = drafts(p, 3, gen)
    check_tree(K, p, q2, dk2, dv2, mask2)
