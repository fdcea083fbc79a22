"""The speculative-decoding operators of the quantised KV cache, as a program calls them:

  rope   rotary positions of queries and keys (forward, and the transposed product that is
         its gradient), out of a fused projection's rows
  read   reading cached keys and values back out of a quantised cache
  tree   attention of a tree of drafted tokens over a quantised cache

With `own` false, run() computes them in elementary torch operations in 32 bits from a
plainly packed copy of the same cache; with `own` true it calls this package.  Tokens are
drawn with the structure of real caches: a few key channels large in every token, a few
value tokens large in all channels.
"""
import math

import torch

own = False

DEVICE = "cuda"
ROWS, FP8 = ("int8", "int4"), ("fp8", "fp8e5m2")


# ------------------------------------------------------------------------------ the cases
def _cache(scheme="kivi", bits=2, group_k=32, group_v=32, residual=128, batch=1, q_heads=32,
           kv_heads=8, head_dim=128, lo=4096, hi=4096, page_groups=0, outliers=0, rope_base=0.0):
    return dict(scheme=scheme, bits=bits, group_k=group_k, group_v=group_v, residual=residual, batch=batch,
                q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, lo=lo, hi=hi, page_groups=page_groups,
                outliers=outliers, rope_base=rope_base)


def _rope(tokens, q_heads, kv_heads, head_dim, rotary_dim, layout, scaling, dtype, transpose, top, base=500000.0,
          factor=8.0, low=1.0, high=4.0, original=8192, magnitude=1.0):
    return dict(op="rope", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                rotary_dim=rotary_dim, layout=layout, scaling=scaling, dtype=dtype, transpose=transpose, top=top,
                base=base, factor=factor, low=low, high=high, original=original, magnitude=magnitude)


def listed():
    return [
        # one decode step of eight conversations: latency
        dict(_rope(8, 32, 8, 128, 128, "half", "by_parts", "bf16", False, 131072), name="rope_step"),
        # a prompt of 16384 tokens, all heads
        dict(_rope(16384, 32, 8, 128, 128, "half", "none", "bf16", False, 16384), name="rope_prompt"),
        # the gradient of a training batch's rotation: half of each head, interleaved, fp32
        dict(_rope(4099, 16, 16, 128, 64, "interleaved", "by_parts", "f32", True, 65536, base=10000.0, factor=16.0,
                   high=32.0, original=4096, magnitude=0.1 * math.log(16.0) + 1.0), name="rope_gradient"),
        # the newest tokens of one conversation out of a dense-and-sparse cache
        dict(_cache(bits=4, group_k=64, group_v=64, outliers=1, lo=1000, hi=1000), op="read", first=743, count=257,
             dtype="bf16", name="read_newest"),
        # a 2-bit layer of eight conversations, whole
        dict(_cache(batch=8), op="read", first=0, count=4096, dtype="bf16", name="read_layer"),
        # an FP8 layer of many conversations, moved out
        dict(_cache("fp8", batch=24, lo=8192, hi=8192), op="read", first=0, count=8192, dtype="bf16",
             name="read_fp8"),
        # a short draft of one short conversation: latency
        dict(_cache(lo=700, hi=700), op="tree", nodes=4, shape="chain", ragged=False, name="tree_short"),
        # the 2-bit layer of eight conversations, 16 drafted tokens each
        dict(_cache(batch=8), op="tree", nodes=16, shape="tree", ragged=False, name="tree_layer"),
        # a long 4-bit context, a tree of 32
        dict(_cache(bits=4, group_k=128, group_v=128, lo=131072, hi=131072), op="tree", nodes=32, shape="tree",
             ragged=False, name="tree_128k"),
        # a serving mix in pages, ragged contexts and drafts
        dict(_cache(batch=48, lo=1024, hi=16384, page_groups=16), op="tree", nodes=11, shape="tree", ragged=True,
             name="tree_serve_paged"),
        # an FP8 batch, eight drafts each
        dict(_cache("fp8", batch=64, lo=8192, hi=8192), op="tree", nodes=8, shape="tree", ragged=False,
             name="tree_fp8"),
        # per-token INT8 rows, narrow heads, eight query heads a KV head, a wide tree
        dict(_cache("int8", batch=5, q_heads=16, kv_heads=2, head_dim=64, lo=1500, hi=9001), op="tree", nodes=61,
             shape="tree", ragged=True, name="tree_int8_wide"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "read", "tree", "tree"])
    if op == "rope":
        D = rng.choice([64, 96, 128, 256])
        R = rng.choice([D, D, D // 2, D // 4])
        g, H = rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
        tokens = max(1, _log(rng, 1, 16384) * 40 * 128 // ((g + 1) * H * D * 2 + 40 * 128))
        scaling = rng.choice(["none", "linear", "ntk", "by_parts"])
        factor = rng.choice([2.0, 4.0, 8.0, 16.0])
        return _rope(tokens, g * H, H, D, R, rng.choice(["half", "interleaved"]), scaling,
                     rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.4, rng.choice([4096, 16384, 131072]),
                     base=rng.choice([10000.0, 500000.0]), factor=factor, high=rng.choice([4.0, 32.0]),
                     original=rng.choice([4096, 8192]), magnitude=rng.choice([1.0, 0.1 * math.log(factor) + 1.0]))
    scheme = rng.choice(["kivi", "kivi", "kivi", "int8", "int4", "fp8", "fp8e5m2"])
    D = rng.choice([64, 128, 128, 256] if scheme == "kivi" else [32, 64, 128, 256])
    g, H = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    kw = dict(scheme=scheme, q_heads=g * H, kv_heads=H, head_dim=D)
    if scheme == "kivi":
        kw.update(bits=rng.choice([2, 2, 4, 4, 8]), group_k=rng.choice([16, 32, 48, 64, 128]),
                  group_v=rng.choice([16, 32, 64]), residual=rng.choice([0, 32, 128, 129]),
                  page_groups=rng.choice([0, 0, 1, 7, 16]), outliers=rng.choice([0, 0, 0, 1, 3]),
                  rope_base=rng.choice([0.0, 0.0, 0.0, 10000.0]))
        if D == 256:                                         # what the decode's tiles hold
            kw.update(bits=min(kw["bits"], 4), outliers=0)
    kw["batch"], nodes = _log(rng, 1, 64), _log(rng, 1, 64)
    # at most a quarter of the largest case's cached values, and its products
    top = min(131072, 64 * 8192 * 8 * 128 // 4 // (kw["batch"] * H * D))
    if op == "tree":
        top = min(top, 64 * 8192 * 32 * 8 * 128 // (kw["batch"] * g * H * D * nodes))
    hi = _log(rng, 16, max(16, top))
    kw.update(lo=rng.choice([hi, max(1, hi // 16)]), hi=hi)
    if scheme == "kivi" and hi - kw["residual"] < kw["group_k"]:
        kw["page_groups"] = 0                                # no packed group: no pages
    c = _cache(**kw)
    if op == "read":
        first = rng.choice([0, rng.randint(0, hi - 1)])
        return dict(c, op="read", first=first, count=rng.randint(1, hi - first), dtype=rng.choice(["bf16", "bf16", "f32"]))
    return dict(c, op="tree", nodes=nodes, shape=rng.choice(["chain", "tree", "tree"]),
                ragged=rng.random() < 0.5)


# ------------------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _keys_values(c, gen, tokens):
    """bf16 keys and values [batch][tokens][kv_heads][head_dim]: four key channels of a head
    8 to 16 times the others, one value token in a hundred 8 times the others."""
    B, H, D = c["batch"], c["kv_heads"], c["head_dim"]
    mult = torch.ones(H, D, device=DEVICE)
    at = torch.rand(H, D, generator=gen, device=DEVICE).argsort(1)[:, :4]
    mult.scatter_(1, at, 8.0 + 8.0 * torch.rand(H, 4, generator=gen, device=DEVICE))
    k = torch.randn(B, tokens, H, D, generator=gen, device=DEVICE).mul_(mult).to(torch.bfloat16)
    v = torch.randn(B, tokens, H, D, generator=gen, device=DEVICE)
    v.mul_(torch.where(torch.rand(B, tokens, 1, 1, generator=gen, device=DEVICE) < 0.01, 8.0, 1.0))
    return k, v.to(torch.bfloat16), mult


def _lengths(c, gen):
    """Tokens of each sequence, the longest `hi`."""
    n = torch.randint(c["lo"], c["hi"] + 1, (c["batch"],), generator=gen, device=DEVICE)
    n[0] = c["hi"]
    return n


def _fp8_scales(c, k, v):
    top = 448.0 if c["scheme"] == "fp8" else 57344.0
    return torch.stack([x.float().abs().amax(dim=(0, 1, 3)) / top for x in (k, v)], dim=1).contiguous()


def _pages(c, gen):
    """(pages in the pool, int64 [batch][pages of a sequence]): shuffled pages of each run of
    `page_groups` groups; one page per group in its own order where the cache has no pages."""
    groups = max(0, c["hi"] - c["residual"]) // c["group_k"]
    each = -(-groups // max(1, c["page_groups"]))
    pool = c["batch"] * each + max(1, c["batch"] * each // 100)
    order = torch.rand(pool, generator=gen, device=DEVICE).argsort()[: c["batch"] * each]
    return pool, (order if c["page_groups"] else torch.arange(c["batch"] * each, device=DEVICE)).view(c["batch"], each)


def _raw(c, seed):
    """Everything the cache cases are made from: the tokens, the counts, the pages."""
    gen = _generator(seed)
    k, v, mult = _keys_values(c, gen, c["hi"])
    n = _lengths(c, gen)
    pool, table = _pages(c, gen) if c["scheme"] == "kivi" else (0, None)
    r = dict(k=k, v=v, n=n, pool=pool, table=table)
    if c["scheme"] in FP8:
        r["scales"] = _fp8_scales(c, k, v)
    if c["op"] == "tree":
        B, T, H, D = c["batch"], c["nodes"], c["kv_heads"], c["head_dim"]
        r["q"] = torch.randn(B, T, c["q_heads"], D, generator=gen, device=DEVICE).to(torch.bfloat16)
        r["dk"] = torch.randn(B, T, H, D, generator=gen, device=DEVICE).mul_(mult).to(torch.bfloat16)
        r["dv"] = torch.randn(B, T, H, D, generator=gen, device=DEVICE).to(torch.bfloat16)
        r["mask"] = _tree_mask(c, gen) if c["shape"] == "tree" else None
        r["nodes"] = None
        if c["ragged"]:
            r["nodes"] = torch.randint(0 if B > 1 else 1, T + 1, (B,), generator=gen, device=DEVICE, dtype=torch.int32)
            r["nodes"][0] = T
    return r


def _tree_mask(c, gen):
    """[batch][nodes][nodes] truth values: node i sees itself and its ancestors.  Node i's
    parent is drawn among the nodes before it (two thirds of them among the last four)."""
    B, T = c["batch"], c["nodes"]
    i = torch.arange(T, device=DEVICE)
    u = torch.rand(B, T, generator=gen, device=DEVICE)
    near = torch.rand(B, T, generator=gen, device=DEVICE) < 0.67
    span = torch.where(near, i.clamp(max=4), i)
    parent = (i - 1 - (u * span).long()).clamp(min=0)
    step = torch.zeros(B, T, T, device=DEVICE).scatter_(2, parent.unsqueeze(2), 1.0)
    step[:, 0] = 0.0
    seen = torch.eye(T, device=DEVICE).expand(B, T, T) + step
    for _ in range(max(1, (T - 1).bit_length())):     # paths of up to 2, 4, 8, ... edges
        seen = (torch.bmm(seen, seen) > 0).float()
    return seen > 0


# ------------------------------------------------------------------------------ the plain cache
def _half_toward(x, up):
    """binary16 of x rounded toward +infinity (up) or -infinity."""
    h = x.to(torch.float16)
    b = h.view(torch.int16).to(torch.int32) & 0xFFFF
    f = h.float()
    if up:
        step = torch.where(f == 0, torch.full_like(b, 0x0001), torch.where(f > 0, b + 1, b - 1))
        b = torch.where(f < x, step, b)
    else:
        step = torch.where(f == 0, torch.full_like(b, 0x8001), torch.where(f > 0, b - 1, b + 1))
        b = torch.where(f > x, step, b)
    return torch.where(b >= 0x8000, b - 0x10000, b).to(torch.int16).view(torch.float16)


def _quantise(x, bits, dim, outliers):
    """Asymmetric codes of the vectors along `dim`: (codes, scale, zero, side values, side
    indices); the side lists hold each vector's elements of largest magnitude."""
    kept = torch.ones_like(x, dtype=torch.bool)
    vals = idx = None
    if outliers:
        size = x.shape[dim]
        place = torch.arange(size, device=x.device).view([-1 if d == dim % x.dim() else 1 for d in range(x.dim())])
        rank = (x.to(torch.bfloat16).view(torch.int16).to(torch.int32) & 0x7FFF) * size + (size - 1 - place)
        idx = rank.topk(outliers, dim=dim).indices
        vals = x.gather(dim, idx).to(torch.bfloat16)
        kept.scatter_(dim, idx, False)
    mn = torch.where(kept, x, math.inf).amin(dim, keepdim=True)
    mx = torch.where(kept, x, -math.inf).amax(dim, keepdim=True)
    z = _half_toward(mn, False)
    # a tensor divisor: a division, where a number's would be a product with its reciprocal
    s = _half_toward((mx - z.float()) / torch.full_like(mx, 2 ** bits - 1), True)
    sf = s.float()
    codes = ((x - z.float()) / torch.where(sf == 0, 1.0, sf)).round().clamp(0, 2 ** bits - 1)
    codes = torch.where((sf == 0) | ~kept, 0.0, codes).to(torch.uint8)
    return codes, s, z, vals, idx


def _pack(codes, bits):
    c = codes.view(*codes.shape[:-1], -1, 8 // bits)
    out = torch.zeros(c.shape[:-1], dtype=torch.uint8, device=c.device)
    for j in range(8 // bits):
        out |= c[..., j] << (bits * j)
    return out


def _plain_cache(c, r):
    """The same cache as plain tensors.  kivi: groups of a pool, [groups][heads][tokens]
    [channels], found through `slot` [batch][groups], and the newest tokens in bf16; int8,
    int4: codes and one scale per token and head; fp8: codes and one scale per head."""
    B, N, H, D = r["k"].shape
    st = {"n": r["n"]}
    if c["scheme"] in FP8:
        t, top = (torch.float8_e4m3fn, 448.0) if c["scheme"] == "fp8" else (torch.float8_e5m2, 57344.0)
        for i, x in enumerate(("k", "v")):
            st[x] = (r[x].float() / r["scales"][:, i].view(1, 1, H, 1)).clamp(-top, top).to(t)
        st["scales"] = r["scales"]
        return st
    if c["scheme"] in ROWS:
        top = 127.0 if c["scheme"] == "int8" else 7.0
        for x in ("k", "v"):
            f = r[x].float()
            s = f.abs().amax(-1, keepdim=True)
            s = s / torch.full_like(s, top)
            code = (f / torch.where(s == 0, 1.0, s)).round().clamp(-top, top).to(torch.int8)
            st[x], st[x + "s"] = code if top > 7 else _pack((code & 15).view(torch.uint8), 4), s
        return st
    G, Gv, R, bits, K = c["group_k"], c["group_v"], c["residual"], c["bits"], c["outliers"]
    n = r["n"]
    st["qn"] = torch.where(n - R >= G, (n - R).clamp(min=0) // G * G, 0)
    NG = max(0, N - R) // G
    PG = max(1, c["page_groups"])
    g = torch.arange(NG, device=DEVICE)
    st["slot"] = r["table"][:, g // PG] * PG + g % PG if NG else torch.zeros(B, 0, dtype=torch.int64, device=DEVICE)
    slots = r["pool"] * PG
    if NG:
        at = st["slot"].reshape(-1)

        def pooled(x):
            x = x.reshape(B * NG, *x.shape[2:])
            return torch.zeros(slots, *x.shape[1:], dtype=x.dtype, device=DEVICE).index_copy_(0, at, x)

        k = r["k"][:, :NG * G].float().view(B, NG, G, H, D).transpose(2, 3)
        code, s, z, val, idx = _quantise(k, bits, 3, K)
        st.update(kq=pooled(_pack(code, bits)), ks=pooled(s.squeeze(3)), kz=pooled(z.squeeze(3)))
        if K:
            st.update(kx=pooled(val), ki=pooled(idx))
        v = r["v"][:, :NG * G].float().view(B, NG, G, H, D).transpose(2, 3).reshape(B, NG, H, G, D // Gv, Gv)
        code, s, z, val, idx = _quantise(v, bits, 5, K)
        st.update(vq=pooled(_pack(code.view(B, NG, H, G, D), bits)), vs=pooled(s), vz=pooled(z))
        if K:
            st.update(vx=pooled(val), vi=pooled(idx))
    recent = (st["qn"].view(B, 1) + torch.arange(min(N, R + G), device=DEVICE)).clamp(max=N - 1)
    b = torch.arange(B, device=DEVICE).view(B, 1)
    st.update(wk=r["k"][b, recent], wv=r["v"][b, recent])
    return st


def _unpacked(x, bits):
    shift = torch.arange(0, 8, bits, device=x.device, dtype=torch.uint8)
    return ((x.unsqueeze(-1) >> shift) & (2 ** bits - 1)).flatten(-2)


def _values(c, st, first, end):
    """fp32 keys and values [batch][tokens][heads][channels] of tokens [first, end)."""
    H, D, at = c["kv_heads"], c["head_dim"], slice(first, end)
    if c["scheme"] in FP8:
        return [st[x][:, at].float() * st["scales"][:, i].view(1, 1, H, 1) for i, x in enumerate(("k", "v"))]
    if c["scheme"] == "int8":
        return [st[x][:, at].float() * st[x + "s"][:, at] for x in ("k", "v")]
    if c["scheme"] == "int4":
        return [((_unpacked(st[x][:, at], 4).to(torch.int8) ^ 8) - 8).float() * st[x + "s"][:, at] for x in ("k", "v")]
    B, G, bits = c["batch"], c["group_k"], c["bits"]
    t = torch.arange(first, end, device=DEVICE)
    late = (t.view(1, -1) - st["qn"].view(B, 1)).clamp(0, st["wk"].shape[1] - 1)
    b = torch.arange(B, device=DEVICE).view(B, 1)
    k, v = st["wk"].float()[b, late], st["wv"].float()[b, late]
    slot = st["slot"][:, first // G:-(-end // G)]
    if slot.shape[1]:
        pk = _unpacked(st["kq"][slot], bits).float() * st["ks"][slot].float().unsqueeze(3) \
            + st["kz"][slot].float().unsqueeze(3)
        pv = _unpacked(st["vq"][slot], bits).float().unflatten(-1, (D // c["group_v"], c["group_v"]))
        pv = pv * st["vs"][slot].float() + st["vz"][slot].float()
        if c["outliers"]:
            pk = pk.scatter(3, st["ki"][slot], st["kx"][slot].float())
            pv = pv.scatter(5, st["vi"][slot], st["vx"][slot].float())
        packed = (t.view(1, -1) < st["qn"].view(B, 1)).view(B, -1, 1, 1)
        here = (t - first // G * G).clamp(max=slot.shape[1] * G - 1)
        k = torch.where(packed, pk.transpose(2, 3).flatten(1, 2)[:, here], k)
        v = torch.where(packed, pv.flatten(4).transpose(2, 3).flatten(1, 2)[:, here], v)
    return [k, v]


# ------------------------------------------------------------------------------ rotary positions
def _frequencies(c):
    """binary32 w_i of the rotation, computed in 64 bits: base^(-2i/R), scaled."""
    R, f = c["rotary_dim"], c["factor"]
    i = torch.arange(R // 2, dtype=torch.float64, device=DEVICE)
    base = c["base"] * f ** (R / (R - 2)) if c["scaling"] == "ntk" else c["base"]
    w = base ** (-2.0 * i / R)
    if c["scaling"] == "linear":
        w = w / f
    if c["scaling"] == "by_parts":
        keep = ((c["original"] * w / (2 * math.pi) - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        w = (1 - keep) * w / f + keep * w
    return w.float()


def _rope_inputs(c, seed):
    """Rows of a fused projection, [tokens][q heads + 2 KV heads][head_dim], and positions."""
    gen = _generator(seed)
    rows = torch.randn(c["tokens"], c["q_heads"] + 2 * c["kv_heads"], c["head_dim"], generator=gen, device=DEVICE)
    rows = rows.to(_dtype(c["dtype"]))
    pos = torch.randint(0, c["top"], (c["tokens"],), generator=gen, device=DEVICE, dtype=torch.int32)
    return rows[:, :c["q_heads"]], rows[:, c["q_heads"]:c["q_heads"] + c["kv_heads"]], pos


def _turned(c, x, cos, sin):
    """x [tokens][heads][head_dim] with the first rotary_dim channels turned, in 32 bits."""
    R = c["rotary_dim"]
    f = x.float()
    a, b = (f[..., :R // 2], f[..., R // 2:R]) if c["layout"] == "half" else (f[..., 0:R:2], f[..., 1:R:2])
    p, q = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([p, q], -1) if c["layout"] == "half" else torch.stack([p, q], -1).flatten(-2)
    return torch.cat([turned, f[..., R:]], -1).to(x.dtype)


# ------------------------------------------------------------------------------ state and pass
def prepare(case, seed):
    c = dict(case)
    if c["op"] == "rope":
        q, k, pos = _rope_inputs(c, seed)
        st = dict(case=c, q=q, k=k, pos=pos)
        if own:
            import quantised_kv_cache_kvq_gb300 as K
            st["rotary"] = K.RotaryEmbedding(c["head_dim"], c["base"], rotary_dim=c["rotary_dim"], layout=c["layout"],
                                             scaling=c["scaling"], factor=c["factor"], low=c["low"], high=c["high"],
                                             original_context=c["original"], magnitude=c["magnitude"])
        else:
            st["w"] = _frequencies(c)
        return st
    r = _raw(c, seed)
    st = dict(case=c)
    if c["op"] == "tree":
        st.update((x, r[x]) for x in ("q", "dk", "dv", "mask", "nodes"))
    if not own:
        st["cache"] = _plain_cache(c, r)
        return st
    import quantised_kv_cache_kvq_gb300 as K
    pages = dict(page_groups=c["page_groups"], num_pages=r["pool"], block_table=r["table"].to(torch.int32).contiguous()) \
        if c["page_groups"] else {}
    st["cache"] = K.QuantizedKVCache(K.make_config(
        c["scheme"], 1, c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"], c["hi"],
        bits=c["bits"] if c["scheme"] == "kivi" else None, group_k=c["group_k"], group_v=c["group_v"],
        residual=c["residual"], rope_base=c["rope_base"], outliers=c["outliers"], **pages))
    st["cache"].append(0, r["k"], r["v"], n_valid=r["n"].to(torch.int32), fp8_scales=r.get("scales"))
    return st


def run(state):
    c = state["case"]
    if c["op"] == "rope":
        return _run_rope(c, state)
    if c["op"] == "read":
        return _run_read(c, state)
    return _run_tree(c, state)


def _run_rope(c, st):
    if own:
        return st["rotary"].rotate(st["q"], st["k"], st["pos"], transpose=c["transpose"])
    # the angle is the binary32 product; its cosine and sine in 64 bits (far positions)
    angle = (st["pos"].float().view(-1, 1, 1) * st["w"]).double()
    cos, sin = (angle.cos() * c["magnitude"]).float(), (angle.sin() * c["magnitude"]).float()
    if c["transpose"]:
        sin = -sin
    return _turned(c, st["q"], cos, sin), _turned(c, st["k"], cos, sin)


def _run_read(c, st):
    if own:
        return st["cache"].read(0, first=c["first"], count=c["count"], dtype=c["dtype"])
    t = torch.arange(c["first"], c["first"] + c["count"], device=DEVICE)
    held = (t.view(1, -1) < st["cache"]["n"].view(-1, 1)).view(c["batch"], -1, 1, 1)
    return tuple(torch.where(held, x, 0.0).to(_dtype(c["dtype"]))
                 for x in _values(c, st["cache"], c["first"], c["first"] + c["count"]))


def _run_tree(c, st):
    if own:
        return st["cache"].tree_decode(0, st["q"], st["dk"], st["dv"], mask=st["mask"], n_nodes=st["nodes"])
    B, T, H, D, N = c["batch"], c["nodes"], c["kv_heads"], c["head_dim"], c["hi"]
    g = c["q_heads"] // H
    k, v = _values(c, st["cache"], 0, N)
    if c["rope_base"]:
        half = D // 2
        w = (c["rope_base"] ** (-2.0 * torch.arange(half, dtype=torch.float64, device=DEVICE) / D)).float()
        angle = (torch.arange(N, device=DEVICE).float().view(N, 1, 1) * w).double()
        cos, sin = angle.cos().float(), angle.sin().float()
        a, b = k[..., :half], k[..., half:]
        k = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    k = torch.cat([k, st["dk"].float()], 1).permute(0, 2, 3, 1)                  # [B][H][D][N + T]
    v = torch.cat([v, st["dv"].float()], 1).transpose(1, 2)                      # [B][H][N + T][D]
    q = st["q"].float().view(B, T, H, g, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * g, D)
    i = torch.arange(T, device=DEVICE)
    nodes = torch.full((B,), T, device=DEVICE) if st["nodes"] is None else st["nodes"]
    live = i.view(1, T) < nodes.view(B, 1)
    drafts = (i.view(1, T, 1) >= i.view(1, 1, T)).expand(B, T, T) if st["mask"] is None else st["mask"]
    drafts = drafts & live.view(B, 1, T)
    cached = (torch.arange(N, device=DEVICE).view(1, 1, N) < st["cache"]["n"].view(B, 1, 1)).expand(B, T, N)
    seen = torch.cat([cached, drafts], 2).repeat_interleave(g, 1).view(B, 1, T * g, N + T)
    s = torch.where(seen, torch.matmul(q, k) * (1.0 / math.sqrt(D)), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0, 1.0, l)
    o = o.view(B, H, T, g, D).permute(0, 2, 1, 3, 4).reshape(B, T, H * g, D)
    return torch.where(live.view(B, T, 1, 1), o, 0.0).to(torch.bfloat16)


# ------------------------------------------------------------------------------ work
def _token_bytes(c, tokens):
    """Cache bytes that `tokens` tokens of one sequence and KV head take."""
    D = c["head_dim"]
    if c["scheme"] in FP8:
        return 2 * D * tokens
    if c["scheme"] in ROWS:
        return (2 * D + 8 if c["scheme"] == "int8" else D + 8) * tokens
    G, Gv, R = c["group_k"], c["group_v"], c["residual"]
    packed = max(0, tokens - R) // G * G
    side = 4 * c["outliers"]
    return packed * (2 * D * c["bits"] / 8 + (4 + side) * D / G + (4 + side) * D / Gv) + (tokens - packed) * 4 * D


def work(case):
    c = dict(case)
    if c["op"] == "rope":
        size = 2 if c["dtype"] == "bf16" else 4
        x = c["tokens"] * (c["q_heads"] + c["kv_heads"])
        return {"bytes": 2 * x * c["head_dim"] * size + 4 * c["tokens"], "flops": 3 * x * c["rotary_dim"]}
    mean = (c["lo"] + c["hi"]) / 2
    H, D, B = c["kv_heads"], c["head_dim"], c["batch"]
    if c["op"] == "read":
        size = 2 if c["dtype"] == "bf16" else 4
        tokens = max(0.0, min(c["count"], mean - c["first"]))
        read = _token_bytes(c, mean) * tokens / mean
        return {"bytes": B * H * (read + 2 * c["count"] * D * size), "flops": 4 * B * H * tokens * D}
    T = c["nodes"] * (0.5 if c["ragged"] and B > 1 else 1.0)
    read = B * H * _token_bytes(c, mean) + B * T * 2 * D * (2 * c["q_heads"] + 2 * H) + B * T * T
    return {"bytes": read, "flops": 4 * D * B * c["q_heads"] * T * (mean + T / 2)}


# ------------------------------------------------------------------------------ in 64 bits
def _values64(c, st, b, h):
    """Keys and values [tokens][channels] of one sequence and head, in 64 bits."""
    if c["scheme"] in FP8:
        return [st[x][b, :, h].to(torch.float64) * st["scales"][h, i].double() for i, x in enumerate(("k", "v"))]
    if c["scheme"] in ROWS:
        got = []
        for x in ("k", "v"):
            code = st[x][b, :, h]
            if c["scheme"] == "int4":
                lo, hi = (code & 15).double(), (code >> 4).double()
                code = torch.stack([lo - 16 * (lo > 7), hi - 16 * (hi > 7)], -1).flatten(-2)
            got.append(code.double() * st[x + "s"][b, :, h].double())
        return got
    N, D, bits, qn = c["hi"], c["head_dim"], c["bits"], int(st["qn"][b])
    k = torch.zeros(N, D, dtype=torch.float64, device=DEVICE)
    v = torch.zeros(N, D, dtype=torch.float64, device=DEVICE)
    held = min(N - qn, st["wk"].shape[1])
    k[qn:qn + held], v[qn:qn + held] = st["wk"][b, :held, h].double(), st["wv"][b, :held, h].double()
    if qn:
        at = st["slot"][b, :qn // c["group_k"]]

        def codes(x):
            return torch.stack([(x.int() // 2 ** (bits * j)) % 2 ** bits for j in range(8 // bits)], -1).flatten(-2).double()

        pk = codes(st["kq"][at, h]) * st["ks"][at, h].double()[:, None] + st["kz"][at, h].double()[:, None]
        gv = c["group_v"]
        pv = codes(st["vq"][at, h]) * st["vs"][at, h].double().repeat_interleave(gv, -1).flatten(-2) \
            + st["vz"][at, h].double().repeat_interleave(gv, -1).flatten(-2)
        if c["outliers"]:
            pk.scatter_(1, st["ki"][at, h], st["kx"][at, h].double())
            pv.view(*pv.shape[:2], D // gv, gv).scatter_(3, st["vi"][at, h], st["vx"][at, h].double())
        k[:qn], v[:qn] = pk.flatten(0, 1), pv.flatten(0, 1)
    return [k, v]


def exact(case, seed):
    c = dict(case)
    if c["op"] == "rope":
        q, k, pos = _rope_inputs(c, seed)
        R, w = c["rotary_dim"], _frequencies(c)
        turn = torch.polar(torch.full((c["tokens"], R // 2), c["magnitude"], dtype=torch.float64, device=DEVICE),
                           (pos.float()[:, None] * w[None]).double() * (-1 if c["transpose"] else 1))
        got = []
        for x in (q, k):
            y = x.double().clone()
            at = torch.arange(R, device=DEVICE).view(2, -1) if c["layout"] == "half" else \
                torch.arange(R, device=DEVICE).view(-1, 2).T
            z = torch.complex(y[..., at[0]], y[..., at[1]]) * turn[:, None]
            y[..., at[0]], y[..., at[1]] = z.real, z.imag
            got.append(y)
        return tuple(got)
    r = _raw(c, seed)
    st = _plain_cache(c, r)
    B, H, D, N = c["batch"], c["kv_heads"], c["head_dim"], c["hi"]
    if c["op"] == "read":
        out = [torch.zeros(B, c["count"], H, D, dtype=torch.float64, device=DEVICE) for _ in range(2)]
        for b in range(B):
            end = min(int(r["n"][b]), c["first"] + c["count"])
            for h in range(H):
                for o, x in zip(out, _values64(c, st, b, h)):
                    if end > c["first"]:
                        o[b, :end - c["first"], h] = x[c["first"]:end]
        return tuple(out)
    T, g = c["nodes"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros(B, T, c["q_heads"], D, dtype=torch.float64, device=DEVICE)
    for b in range(B):
        n, t = int(r["n"][b]), T if r["nodes"] is None else int(r["nodes"][b])
        if t == 0:
            continue
        see = torch.ones(t, t, dtype=torch.bool, device=DEVICE).tril() if r["mask"] is None else r["mask"][b, :t, :t]
        see = torch.cat([torch.ones(t, n, dtype=torch.bool, device=DEVICE), see], 1)
        for h in range(H):
            k, v = (x[:n] for x in _values64(c, st, b, h))
            if c["rope_base"]:
                w = torch.tensor([c["rope_base"] ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64).float()
                angle = (torch.arange(n).float()[:, None] * w[None]).double().to(DEVICE)
                z = torch.complex(k[:, :D // 2].contiguous(), k[:, D // 2:].contiguous()) * torch.polar(torch.ones_like(angle), angle)
                k = torch.cat([z.real, z.imag], 1)
            k = torch.cat([k, r["dk"][b, :t, h].double()])
            v = torch.cat([v, r["dv"][b, :t, h].double()])
            for j in range(g):
                s = (r["q"][b, :t, h * g + j].double() @ k.T) / math.sqrt(D)
                out[b, :t, h * g + j] = torch.softmax(s.masked_fill(~see, -math.inf), 1).nan_to_num(0.0) @ v
    return out
