"""Cases that measure the 4-bit KV cache (append, decode attention) and the page
operations of paged caches (reserve, fork, compact), with their plain forms.

A 4-bit cache row holds one token of one kv head, K and V together, in groups of 32
dims: per group m = the smallest value rounded down to bf16, s = (largest - m) / 15
rounded up to bf16, and codes rint((x - m) / s) in 0..15; a value stands for
code * s + m.  Bytes of a row: K codes (d/2), K (m, s) bf16 pairs (d/8), V codes, V
pairs.  Codes are 32-bit words in the order [dim % 32 / 8][dim / 32], nibble dim % 8.

Page operations: ref[block] counts the table entries that name a block (0: free).
"""
import math

import torch

own = False

DEV = "cuda"
I32, I64 = torch.int32, torch.int64


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode token of a 32-sequence batch into full rings of a 128-token window
        dict(name="append4_step", op="append", kind="ring", B=32, T=1, Hq=32, Hkv=8, D=128, S=4, W=128, theta=5e5,
             io="bf16"),
        # the long prompt of one sequence into a global layer, all of it kept
        dict(name="append4_prompt", op="append", kind="global", B=1, T=32768, Hq=32, Hkv=8, D=128, S=0, W=0,
             theta=5e5, io="bf16"),
        # the smallest cache: one sequence, six slots, fp32 (latency)
        dict(name="decode4_tiny", op="decode", kind="ring", B=1, Hq=8, Hkv=4, D=64, S=2, W=4, N=6, io="f32",
             sink=False),
        # the windowed layer of a decode step, every ring full
        dict(name="decode4_window", op="decode", kind="ring", B=32, Hq=32, Hkv=8, D=128, S=4, W=4092, N=4096,
             io="bf16", sink=False),
        # two long dialogs on a global layer: the sequence axis is split over the GPU
        dict(name="decode4_long", op="decode", kind="global", B=2, Hq=32, Hkv=8, D=128, S=0, W=0, N=131072,
             io="bf16", sink=False),
        # ragged requests in 16-token pages, window and sinks, learned sink logits
        dict(name="decode4_paged", op="decode", kind="paged", B=32, Hq=32, Hkv=8, D=128, S=4, W=4092, N=8191,
             bs=16, io="bf16", sink=True),
        # before a decode step of 32 requests: a page for every sixteenth, copies where beams share one
        dict(name="reserve_step", op="reserve", B=32, MB=512, bs=16, NB=8192, L=1, Hkv=8, D=128, S=4, W=4092,
             most_new=1, share=4),
        # prompts of up to 2048 tokens for 256 requests: thousands of pages at once
        dict(name="reserve_prompts", op="reserve", B=256, MB=1024, bs=16, NB=65536, L=1, Hkv=1, D=64, S=0, W=0,
             most_new=2048, share=1),
        # four beams of one request change places
        dict(name="fork_beams", op="fork", B=4, MB=64, bs=16, NB=512, L=1),
        # 256 beams (64 requests of 4) over 32 layers, long tables
        dict(name="fork_batch", op="fork", B=256, MB=2048, bs=16, NB=262144, L=32),
        # a small pool of one layer
        dict(name="compact_small", op="compact", B=16, MB=32, bs=16, NB=512, L=1, Hkv=4, D=128, live=0.5),
        # a pool of eight layers, two thirds in use and scattered
        dict(name="compact_pool", op="compact", B=64, MB=128, bs=16, NB=8192, L=8, Hkv=8, D=128, live=0.66),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "reserve", "fork", "compact"])
    if op == "append":
        D, kind = rng.choice([64, 128]), rng.choice(["ring", "global"])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4])
        B = _log(rng, 1, 32)
        T = _log(rng, 1, 32768 // B)
        S, W = (rng.choice([0, 1, 4]), _log(rng, 1, min(8192, 32768 // B))) if kind == "ring" else (0, 0)
        return dict(op=op, kind=kind, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, S=S, W=W, theta=rng.choice([1e4, 5e5]),
                    io=rng.choice(["bf16", "bf16", "f32"]))
    if op == "decode":
        D, kind = rng.choice([64, 128]), rng.choice(["ring", "global", "paged"])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 8])
        B = _log(rng, 1, 64)
        N = _log(rng, 1, min(131072, (1 << 21) // (B * Hkv)))
        S = rng.choice([0, 1, 4, 16])
        W = max(1, N - S) if kind == "ring" else (0 if kind == "global" else rng.choice([0, _log(rng, 1, N)]))
        c = dict(op=op, kind=kind, B=B, Hq=Hq, Hkv=Hkv, D=D, S=S, W=W, N=N, io=rng.choice(["bf16", "bf16", "f32"]),
                 sink=rng.random() < 0.5)
        if kind == "paged":
            c["bs"] = rng.choice([4, 8, 16, 32, 64, 256])
        return c
    if op == "reserve":
        B, bs = _log(rng, 1, 256), rng.choice([8, 16, 32])
        MB = _log(rng, 4, 1024)
        window = rng.random() < 0.5
        return dict(op=op, B=B, MB=MB, bs=bs, NB=_log(rng, 64, 65536), L=rng.choice([1, 2]), Hkv=1, D=64,
                    S=4 if window else 0, W=_log(rng, 1, MB * bs) if window else 0,
                    most_new=_log(rng, 1, 2048), share=rng.choice([1, 2, 4]))
    if op == "fork":
        return dict(op=op, B=_log(rng, 1, 256), MB=_log(rng, 1, 2048), bs=16, NB=_log(rng, 64, 262144),
                    L=rng.choice([1, 8, 32]))
    return dict(op=op, B=_log(rng, 1, 64), MB=_log(rng, 4, 256), bs=rng.choice([8, 16]), NB=_log(rng, 64, 8192),
                L=_log(rng, 1, 8), Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]),
                live=rng.uniform(0.05, 0.95))


# ---------------------------------------------------------------------------
# The 4-bit rows, in elementary operations
# ---------------------------------------------------------------------------

def _io(c):
    return torch.bfloat16 if c["io"] == "bf16" else torch.float32


def _down16(x):
    """x (float32) rounded down to a bf16 value."""
    b = x.view(I32)
    return torch.where(b >= 0, b & -65536, (b + 0xFFFF) & -65536).view(torch.float32)


def _up16(x):
    """x >= 0 (float32) rounded up to a bf16 value."""
    return ((x.view(I32) + 0xFFFF) & -65536).view(torch.float32)


def _quantise(x):
    """x float32 [..., D] -> codes [..., D/32, 32] (float32 whole numbers), s, m [..., D/32, 1]."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    m = _down16(g.amin(-1, keepdim=True))
    s = _up16(((g.amax(-1, keepdim=True) - m).double() / 15).float())   # in 64 bits: it may fall on a bf16 value
    codes = torch.where(s > 0, torch.round((g - m) / torch.where(s > 0, s, 1.0)), 0.0).clamp(0, 15)
    return codes, s, m


def _values(codes, s, m):
    return (codes * s + m).flatten(-2)


def _pack_half(codes, s, m):
    """Codes then (m, s) pairs of K or of V, as bytes."""
    w = codes.to(I64).reshape(*codes.shape[:-1], 4, 8)                       # [..., grp, t, nibble]
    w = (w << (4 * torch.arange(8, device=w.device))).sum(-1).transpose(-1, -2).contiguous()   # [..., t, grp]
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).to(I32).flatten(-2)
    pairs = torch.cat([m, s], -1).flatten(-2).to(torch.bfloat16)
    return [w.view(torch.uint8), pairs.contiguous().view(torch.uint8)]


def _pack(k, v):
    return torch.cat(_pack_half(*_quantise(k)) + _pack_half(*_quantise(v)), -1)


def _unpack_half(codes, pairs):
    ng = codes.shape[-1] // 16
    n = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 4, ng, 8)   # [..., t, grp, nibble]
    n = n.transpose(-3, -2).reshape(*codes.shape[:-1], ng, 32).float()
    p = pairs.contiguous().view(torch.bfloat16).float().reshape(*pairs.shape[:-1], ng, 2)
    return _values(n, p[..., 1:], p[..., :1])


def _unpack(rows):
    """Rows as bytes [..., 5 d / 4] -> K, V float32 [..., d]."""
    d = rows.shape[-1] * 4 // 5
    kc, kp, vc, vp = torch.split(rows, [d // 2, d // 8, d // 2, d // 8], -1)
    return _unpack_half(kc, kp), _unpack_half(vc, vp)


def _rows(shape, D, gen):
    """Packed rows of N(0, 1) keys and values, made a slab at a time."""
    n = math.prod(shape)
    out = torch.empty(n, D * 5 // 4, dtype=torch.uint8, device=DEV)
    for i in range(0, n, 1 << 18):
        k = torch.randn(min(1 << 18, n - i), D, device=DEV, generator=gen).bfloat16().float()
        v = torch.randn(min(1 << 18, n - i), D, device=DEV, generator=gen).bfloat16().float()
        out[i:i + (1 << 18)] = _pack(k, v)
    return out.view(*shape, D * 5 // 4)


# ---------------------------------------------------------------------------
# append: RoPE on q and k in place, then k and v into the cache rows
# ---------------------------------------------------------------------------

MAX_POS = 65536


def _prepare_append(c, gen):
    B, T, D, Hkv = c["B"], c["T"], c["D"], c["Hkv"]
    ring = c["kind"] == "ring"
    cap = c["S"] + c["W"] if ring else T
    io = _io(c)
    st = {"c": c}
    for name, H in (("q", c["Hq"]), ("k", Hkv), ("v", Hkv)):
        st[name] = torch.randn(B, T, H, D, device=DEV, generator=gen).to(io)
    st["rows"] = _rows((B, Hkv, cap), D, gen) if ring else torch.zeros(B, Hkv, cap, D * 5 // 4, dtype=torch.uint8,
                                                                     device=DEV)
    # positions, write index and count of every sequence in one buffer: each pass starts from the same state
    book = torch.zeros(B * 16, dtype=torch.uint8, device=DEV)
    pos, head, count = book[:8 * B].view(I64), book[8 * B:12 * B].view(I32), book[12 * B:].view(I32)
    if ring:
        full = c["S"] + c["W"]
        pos.copy_(torch.randint(full, max(full, 32768) + 1, (B,), device=DEV, generator=gen))
        head.copy_(torch.randint(0, c["W"], (B,), device=DEV, generator=gen))
        count.fill_(c["W"])
    st.update(pos=pos, head=head, count=count, book=book, book0=book.clone())
    # plain form: the cache as the values that it stands for, one more row for tokens that a long chunk drops
    st["kc"], st["vc"] = (torch.cat([x, x[:, :, :1]], 2).bfloat16() for x in _unpack(st["rows"]))
    half = D // 2
    w = c["theta"] ** (-2 * torch.arange(half, dtype=torch.float64, device=DEV) / D)
    a = torch.arange(MAX_POS, dtype=torch.float64, device=DEV)[:, None] * w
    st["cos"], st["sin"] = a.cos().float(), a.sin().float()
    if own:
        import sink_kv_attention_gb300 as sk
        st["sk"] = sk
        st["table"] = sk.RopeTable(D, D, c["theta"], MAX_POS)
        st["layer"] = sk.KVLayer(sk.SK_LAYER_RING if ring else sk.SK_LAYER_GLOBAL, st["rows"], None, pos, c["S"],
                                 c["W"], head if ring else None, count if ring else None, None,
                                 torch.zeros(1, dtype=I32, device=DEV))
    return st


def _slots(c, pos, head):
    """Cache slot of each token [B, T]; the row after the last for a dropped one."""
    t = torch.arange(c["T"], device=DEV)
    P = pos[:, None] + t
    if c["kind"] == "global":
        return P
    S, W = c["S"], c["W"]
    t0 = (S - pos).clamp(0, c["T"])[:, None]
    n, u = c["T"] - t0, t - t0
    long = torch.where(u >= n - W, S + u - (n - W), S + W)
    return torch.where(P < S, P, torch.where(n >= W, long, S + (head[:, None] + u) % W))


def _state_after(c, pos, head, count):
    if c["kind"] == "global":
        return pos + c["T"], head, count
    n = c["T"] - (c["S"] - pos).clamp(0, c["T"])
    full = n >= c["W"]
    return (pos + c["T"], torch.where(full, 0, (head + n) % c["W"]).to(I32),
            torch.where(full, c["W"], (count + n).clamp(max=c["W"])).to(I32))


def _rotate(x, cos, sin):
    """x [B, T, H, D], cos and sin [B, T, D/2], in their type."""
    x1, x2 = x.chunk(2, -1)
    cos, sin = cos[:, :, None], sin[:, :, None]
    return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)


def _run_append(st):
    c = st["c"]
    if own:
        sk, layer = st["sk"], st["layer"]
        st["book"].copy_(st["book0"])
        sk.kv_append(st["table"], layer, st["q"], st["k"], st["v"])
        K, V = sk.kv4_unpack(layer.k)
        return [st["q"], st["k"], K, V, layer.pos, st["head"], st["count"]]
    st["book"].copy_(st["book0"])
    pos, head, count = st["pos"], st["head"], st["count"]
    P = pos[:, None] + torch.arange(c["T"], device=DEV)
    cos, sin = st["cos"][P].double(), st["sin"][P].double()
    for name in ("q", "k"):
        st[name].copy_(_rotate(st[name].double(), cos, sin))
    slot = _slots(c, pos, head)
    b = torch.arange(c["B"], device=DEV)[:, None]
    for name, cache in (("k", "kc"), ("v", "vc")):
        st[cache][b, :, slot] = _values(*_quantise(st[name].float())).to(st[cache].dtype)
    pos2, head2, count2 = _state_after(c, pos, head, count)
    return [st["q"], st["k"], st["kc"][:, :, :-1], st["vc"][:, :, :-1], pos2, head2, count2]


def _exact_append(c, seed):
    st = _prepare_append(c, torch.Generator(DEV).manual_seed(seed))
    P = st["pos"][:, None] + torch.arange(c["T"], device=DEV)
    half = c["D"] // 2
    w = c["theta"] ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    z = torch.polar(torch.ones_like(P, dtype=torch.float64)[..., None].expand(*P.shape, half), P[..., None] * w)
    out = []
    for name in ("q", "k"):
        x = st[name].double()
        r = torch.complex(x[..., :half], x[..., half:]) * z[:, :, None]
        out.append(torch.cat([r.real, r.imag], -1))
    k, v = out[1].to(_io(c)).float(), st["v"].float()   # the cache keeps the key that k is left with
    slot = _slots(c, st["pos"], st["head"])
    for new, old in ((k, "kc"), (v, "vc")):
        x = new.double().unflatten(-1, (-1, 32))
        lo = _down16(x.amin(-1).float()).double()
        s = ((x.amax(-1) - lo) / 15).float()
        s = _up16(s).double()
        y = torch.floor((x - lo[..., None]) / s[..., None].clamp(min=1e-300))
        r = (x - lo[..., None]) / s[..., None].clamp(min=1e-300) - y
        y = y + ((r > 0.5) | ((r == 0.5) & (y % 2 == 1)))
        y = (y.clamp(0, 15) * s[..., None] + lo[..., None]).flatten(-2)
        full = st[old].double()
        full[torch.arange(c["B"], device=DEV)[:, None], :, slot] = y
        out.append(full[:, :, :-1])
    return out + [None, None, None]


def _work_append(c):
    e = 2 if c["io"] == "bf16" else 4
    rows = c["B"] * c["T"] * c["D"] * e
    cap = c["S"] + c["W"] if c["kind"] == "ring" else c["T"]
    stored = c["B"] * min(c["T"], cap) * c["Hkv"] * c["D"] * 5 // 4
    values = 2 * c["B"] * c["Hkv"] * cap * c["D"] * 2                         # the cache, returned as values
    held = c["B"] * c["Hkv"] * cap * c["D"] * 5 // 4
    return {"bytes": rows * (2 * c["Hq"] + 3 * c["Hkv"]) + stored + held + values,
            "flops": c["B"] * c["T"] * c["D"] * (3 * c["Hq"] + 9 * c["Hkv"])}


# ---------------------------------------------------------------------------
# decode: one query per sequence over the visible rows of a 4-bit cache
# ---------------------------------------------------------------------------

def _prepare_decode(c, gen):
    B, Hkv, D, N = c["B"], c["Hkv"], c["D"], c["N"]
    st = {"c": c}
    st["q"] = (torch.randn(B, c["Hq"], D, device=DEV, generator=gen)).to(_io(c))
    st["sink"] = torch.randn(c["Hq"], device=DEV, generator=gen) if c["sink"] else None
    err = torch.zeros(1, dtype=I32, device=DEV)
    if c["kind"] == "paged":
        # request lengths from 1 to N; pages in no order
        lens = torch.randint(1, N + 1, (B,), device=DEV, generator=gen)
        lens[0] = N
        bs = c["bs"]
        MB = -(-N // bs)
        st["table"] = torch.randperm(B * MB, device=DEV, generator=gen).to(I32).view(B, MB)
        st["rows"] = _rows((B * MB, Hkv, bs), D, gen)
        st["lens"] = lens
    else:
        S, ring = c["S"], c["kind"] == "ring"
        cap = S + c["W"] if ring else N
        st["rows"] = _rows((B, Hkv, cap), D, gen)
        st["head"] = torch.zeros(B, dtype=I32, device=DEV)
        st["count"] = torch.zeros(B, dtype=I32, device=DEV)
        if ring:   # full rings at a position of their own
            st["lens"] = torch.randint(cap, max(cap, 32768) + 1, (B,), device=DEV, generator=gen)
            st["head"].copy_(torch.randint(0, c["W"], (B,), device=DEV, generator=gen))
            st["count"].fill_(c["W"])
        else:      # prefixes from half the capacity up, the first one full
            st["lens"] = torch.randint(N // 2 + 1, N + 1, (B,), device=DEV, generator=gen)
            st["lens"][0] = N
    if own:
        import sink_kv_attention_gb300 as sk
        st["sk"] = sk
        if c["kind"] == "paged":
            st["layer"] = sk.PagedLayer(st["rows"], None, st["table"], None, st["lens"], err, c["S"], c["W"])
        else:
            st["layer"] = sk.KVLayer(sk.SK_LAYER_RING if ring else sk.SK_LAYER_GLOBAL, st["rows"], None, st["lens"],
                                     c["S"], c["W"], st["head"], st["count"], None, err)
    return st


def _visible(st):
    """Rows [B, Hkv, n, bytes] that hold every visible key, and which of them are visible [B, n]."""
    c = st["c"]
    if c["kind"] != "paged":
        n = st["rows"].shape[2]
        last = st["lens"] if c["kind"] == "global" else st["lens"].clamp(max=c["S"]) + st["count"]
        return st["rows"], torch.arange(n, device=DEV) < last[:, None]
    L, S, W, bs = st["lens"][:, None], c["S"], c["W"], c["bs"]
    most = c["N"] if W <= 0 else min(c["N"], S + W)
    r = torch.arange(most, device=DEV)[None]
    key = torch.where((r >= S) & (L > S + W), L - W + (r - S), r) if W > 0 else r.expand(L.shape[0], -1)
    ok = key < L
    key = torch.where(ok, key, 0)
    block = st["table"].gather(1, key // bs).long()
    return st["rows"][block, :, key % bs].transpose(1, 2), ok


def _run_decode(st):
    c = st["c"]
    if own:
        f = st["sk"].paged_decode_attention if c["kind"] == "paged" else st["sk"].decode_attention
        return f(st["layer"], st["q"], sink_logits=st["sink"])
    rows, ok = _visible(st)
    K, V = _unpack(rows)
    B, Hkv, _, D = K.shape
    q = st["q"].float().view(B, Hkv, -1, D)
    s = (q @ K.transpose(-1, -2)) / math.sqrt(D)
    s = s.masked_fill(~ok[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    z = None
    if st["sink"] is not None:
        z = st["sink"].clamp(-10, 15).view(1, Hkv, -1, 1)
        top = torch.maximum(top, z)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True) + (0 if z is None else torch.exp(z - top))
    return ((p @ V) / total).view(B, -1, D).to(st["q"].dtype)


def _exact_decode(c, seed):
    st = _prepare_decode(c, torch.Generator(DEV).manual_seed(seed))
    rows, ok = _visible(st)
    B, Hkv, n, _ = rows.shape
    D, rep = c["D"], c["Hq"] // c["Hkv"]
    dims = torch.arange(D, device=DEV)
    at = (dims % 32 // 8 * (D // 32) + dims // 32) * 4 + dims % 8 // 2     # byte of each dim's code
    out = torch.empty(B, c["Hq"], D, dtype=torch.float64, device=DEV)
    for b in range(B):
        for g in range(Hkv):
            x = rows[b, g][ok[b]]
            half = []
            for o in (0, D * 5 // 8):
                code = (x[:, o + at] >> (4 * (dims % 2)).to(torch.uint8)) & 15
                par = x[:, o + D // 2:o + D * 5 // 8].contiguous().view(torch.bfloat16).double()
                half.append(code.double() * par[:, 1::2][:, dims // 32] + par[:, 0::2][:, dims // 32])
            q = st["q"][b, g * rep:(g + 1) * rep].double()
            s = q @ half[0].T / D ** 0.5
            if st["sink"] is not None:
                z = st["sink"][g * rep:(g + 1) * rep].double().clamp(-10, 15)
                s = torch.cat([s, z[:, None]], 1)
                w = torch.softmax(s, 1)[:, :-1]
            else:
                w = torch.softmax(s, 1)
            out[b, g * rep:(g + 1) * rep] = w @ half[1]
    return out


def _work_decode(c):
    # rows that are visible: full rings; prefixes of 3/4 of the capacity, requests of half of it on average
    if c["kind"] == "ring":
        rows = c["B"] * (c["S"] + c["W"])
    elif c["kind"] == "global":
        rows = c["N"] + (c["B"] - 1) * 3 * c["N"] / 4
    else:
        m, cap = c["N"], c["N"] if c["W"] <= 0 else min(c["N"], c["S"] + c["W"])
        rows = cap + (c["B"] - 1) * (cap / 2 * cap / m + cap * (1 - cap / m))
    e = 2 if c["io"] == "bf16" else 4
    return {"bytes": rows * c["Hkv"] * c["D"] * 5 / 4 + 2 * c["B"] * c["Hq"] * c["D"] * e,
            "flops": 4 * rows * c["Hq"] * c["D"]}


# ---------------------------------------------------------------------------
# Page operations
# ---------------------------------------------------------------------------

def _book(B, MB, NB):
    """Block table [B, MB] and reference counts [NB] in one buffer, put back before each pass."""
    book = torch.full((B * MB + NB,), -1, dtype=I32, device=DEV)
    return book, book[:B * MB].view(B, MB), book[B * MB:]


def _fill_tables(table, ref, pages, share, gen):
    """Row b takes pages[b] pages in shuffled order; each run of `share` rows is one request's
    beams, which hold the same pages but for the first row's."""
    B, MB = table.shape
    NB = ref.numel()
    j = torch.arange(MB, device=DEV)
    owner = torch.arange(B, device=DEV) // share * share
    pages = pages[owner]
    first = torch.arange(B, device=DEV) == owner
    start = (pages * first).cumsum(0) - pages * first
    perm = torch.randperm(NB, device=DEV, generator=gen).to(I32)
    at = start[owner][:, None] + j
    has = (j < pages[:, None]) & (at < NB)
    table.copy_(torch.where(has, perm[at.clamp(max=NB - 1)], -1))
    ref.zero_()
    ref.scatter_add_(0, torch.where(has, table, 0).flatten().long(), has.flatten().to(I32))
    return has.sum(1)


def _pools(c, gen):
    """K and V pools of every layer; a page more than the layers see, which the plain form
    uses for copies that are none."""
    return torch.randn(2, c["L"], c["NB"] + 1, c["Hkv"], c["bs"], c["D"], device=DEV, generator=gen,
                       dtype=torch.bfloat16)


def _group(c, st, pools):
    import sink_kv_attention_gb300 as sk
    NB = c["NB"]
    err = torch.zeros(1, dtype=I32, device=DEV)
    layers = [sk.PagedLayer(pools[0, i, :NB], pools[1, i, :NB], st["table"], None, st["lens"][i], err, c.get("S", 0),
                            c.get("W", 0)) for i in range(c["L"])]
    return sk.PagedGroup(layers, ref=st["ref"])


def _prepare_reserve(c, gen):
    B, MB, NB, bs = c["B"], c["MB"], c["NB"], c["bs"]
    st = {"c": c}
    st["book"], st["table"], st["ref"] = _book(B, MB, NB)
    # what each request holds before: a part of its fair share of the pool
    most = max(1, min(MB - 1, NB * c["share"] // (2 * B)))
    pages = torch.randint(0, most + 1, (B,), device=DEV, generator=gen)
    held = _fill_tables(st["table"], st["ref"], pages, c["share"], gen)
    # the last held page is filled in part, or whole
    lens = (held * bs - torch.randint(0, bs, (B,), device=DEV, generator=gen)).clamp(min=0)
    owner = torch.arange(B, device=DEV) // c["share"] * c["share"]
    st["lens"] = lens[owner].repeat(c["L"], 1)
    st["n_new"] = torch.randint(1, c["most_new"] + 1, (B,), device=DEV, generator=gen).to(I32)
    st["book0"] = st["book"].clone()
    st["pools"] = _pools(c, gen)
    if own:
        st["group"] = _group(c, st, st["pools"])
    return st


def _run_reserve(st):
    c = st["c"]
    if own:
        st["book"].copy_(st["book0"])
        granted = st["group"].reserve(st["n_new"])
        return [st["table"], st["ref"], granted, st["pools"][:, :, :c["NB"]]]
    B, MB, NB, bs = c["B"], c["MB"], c["NB"], c["bs"]
    table, ref = st["book0"][:B * MB].view(B, MB).long(), st["book0"][B * MB:].long()
    lens, n = st["lens"][0], st["n_new"].long()
    j = torch.arange(MB, device=DEV)
    valid = (table >= 0) & (table < NB)
    if c["W"] > 0:   # pages that the window has left
        keep = lens + n.clamp(max=1) - c["W"]
        dead = valid & ((j + 1) * bs <= keep[:, None]) & (j * bs >= c["S"])
        ref = ref.scatter_add(0, torch.where(dead, table, 0).flatten(), -dead.flatten().long())
        table = torch.where(dead, -1, table)
        valid = valid & ~dead
    first, last = lens // bs, (lens + n - 1) // bs
    over = lens + n > MB * bs
    part = (lens % bs > 0) & ~over
    entry = table.gather(1, first.clamp(max=MB - 1)[:, None])[:, 0]
    bad = part & ((entry < 0) | (entry >= NB))
    ok = (n > 0) & ~bad & ~over
    want = ok[:, None] & (j >= first[:, None]) & (j <= last[:, None])
    shared = valid & (ref[torch.where(valid, table, 0)] > 1)
    alloc = want & (~valid | shared)
    # a shared page that is filled in part is copied; the last of its holders keeps it if all of them write
    copy = part & ok & shared.gather(1, first.clamp(max=MB - 1)[:, None])[:, 0]
    e = torch.where(copy, entry, NB)
    writers = torch.zeros(NB + 1, dtype=I64, device=DEV).scatter_add(0, e, copy.long())
    row = torch.arange(B, device=DEV)
    latest = torch.full((NB + 1,), -1, dtype=I64, device=DEV).scatter_reduce(0, e, row, "amax")
    refs = torch.cat([ref, ref.new_zeros(1)])
    keeper = copy & (writers[e] == refs[e]) & (latest[e] == row)
    copy = copy & ~keeper
    alloc = alloc & ~(keeper[:, None] & (j == first[:, None]))
    granted = (n <= 0) | (ok & (alloc.sum(1).cumsum(0) <= (ref == 0).sum()))
    alloc = alloc & granted[:, None]
    copy = copy & granted
    free = torch.argsort((ref != 0).long(), stable=True)
    rank = (alloc.flatten().long().cumsum(0) - 1).clamp(0, NB - 1).view(B, MB)
    new = torch.where(alloc, free[rank], NB)
    gone = alloc & shared
    ref = ref.scatter_add(0, torch.where(gone, table, 0).flatten(), -gone.flatten().long())
    ref = torch.cat([ref, ref.new_zeros(1)]).scatter(0, new.flatten(), 1)[:NB]
    src = torch.where(copy, entry, NB)
    dst = torch.where(copy, new.gather(1, first.clamp(max=MB - 1)[:, None])[:, 0], NB)
    st["pools"][:, :, dst] = st["pools"][:, :, src]
    table = torch.where(alloc, new, table)
    return [table.to(I32), ref.to(I32), granted.to(I32), st["pools"][:, :, :NB]]


def _work_reserve(c):
    page = 2 * c["L"] * c["Hkv"] * c["bs"] * c["D"] * 2
    copies = c["B"] * (c["share"] - 1) / c["share"] * (1 - 1 / c["bs"])
    return {"bytes": 2 * page * copies + 8 * c["B"] * c["MB"] + 8 * c["NB"] + 20 * c["B"], "flops": 0}


def _prepare_fork(c, gen):
    B, MB, NB = c["B"], c["MB"], c["NB"]
    st = {"c": c}
    st["book"], st["table"], st["ref"] = _book(B, MB, NB)
    pages = torch.randint(0, max(1, min(MB, NB // B)) + 1, (B,), device=DEV, generator=gen)
    held = _fill_tables(st["table"], st["ref"], pages, 1, gen)
    # beam search: every row goes on from one of its request's four rows; a few requests end
    row = torch.arange(B, device=DEV)
    parents = (row // 4 * 4 + torch.randint(0, 4, (B,), device=DEV, generator=gen)).clamp(max=B - 1)
    ended = torch.rand(B, device=DEV, generator=gen) < 0.05
    st["parents"] = torch.where(ended, -1, parents).to(I32)
    tokens = (held * c["bs"] - torch.randint(0, c["bs"], (B,), device=DEV, generator=gen)).clamp(min=0)
    st["lens"] = tokens.repeat(c["L"], 1)
    st["book0"], st["lens0"] = st["book"].clone(), st["lens"].clone()
    if own:
        st["group"] = _group(c, st, _small_pools(c))
    return st


def _small_pools(c):
    """Pools that a fork never touches: one buffer for all layers."""
    one = torch.zeros(1, 1, c["NB"], 1, c["bs"], 64, device=DEV, dtype=torch.bfloat16)
    return one.expand(2, c["L"], -1, -1, -1, -1)


def _run_fork(st):
    c = st["c"]
    if own:
        st["book"].copy_(st["book0"])
        st["lens"].copy_(st["lens0"])
        st["group"].fork(st["parents"])
        return [st["table"], st["ref"], st["lens"]]
    B, MB, NB = c["B"], c["MB"], c["NB"]
    table, ref = st["book0"][:B * MB].view(B, MB).long(), st["book0"][B * MB:]
    parents = st["parents"].long()
    gone = parents < 0
    new = torch.where(gone[:, None], -1, table[parents.clamp(min=0)])
    for t, sign in ((table, -1), (new, 1)):
        ok = (t >= 0) & (t < NB)
        ref = ref.scatter_add(0, torch.where(ok, t, 0).flatten(), (sign * ok).flatten().to(I32))
    lens = torch.where(gone, 0, st["lens0"][:, parents.clamp(min=0)])
    return [new.to(I32), ref, lens]


def _work_fork(c):
    return {"bytes": 8 * c["B"] * c["MB"] + 8 * c["NB"] + 16 * c["B"] * c["L"] + 4 * c["B"], "flops": 0}


def _prepare_compact(c, gen):
    B, MB, NB = c["B"], c["MB"], c["NB"]
    st = {"c": c}
    st["book"], st["table"], st["ref"] = _book(B, MB, NB)
    each = max(1, min(MB, int(NB * c["live"]) // B))
    pages = torch.full((B,), each, dtype=I64, device=DEV)
    held = _fill_tables(st["table"], st["ref"], pages, 1, gen)
    st["lens"] = (held * c["bs"]).repeat(c["L"], 1)
    st["book0"] = st["book"].clone()
    st["pools"] = _pools(c, gen)
    if own:
        st["group"] = _group(c, st, st["pools"])
    return st


def _run_compact(st):
    c = st["c"]
    if own:
        st["book"].copy_(st["book0"])
        block_map, used = st["group"].compact()
        return [st["table"], st["ref"], block_map, used, st["pools"][:, :, :c["NB"]]]
    B, MB, NB = c["B"], c["MB"], c["NB"]
    table, ref = st["book0"][:B * MB].view(B, MB).long(), st["book0"][B * MB:].long()
    live = ref > 0
    n = live.sum()
    ids = torch.arange(NB, device=DEV)
    mover, hole = live & (ids >= n), ~live & (ids < n)
    # the k-th live page behind the first n goes to the k-th free one among them
    kth = torch.full((NB + 1,), NB, dtype=I64, device=DEV).scatter(
        0, torch.where(hole, hole.long().cumsum(0) - 1, NB), ids)
    to = torch.where(mover, kth[(mover.long().cumsum(0) - 1).clamp(0, NB)], torch.where(live, ids, -1))
    dst, src = torch.where(mover, to, NB), torch.where(mover, ids, NB)
    st["pools"][:, :, dst] = st["pools"][:, :, src]
    ref = torch.where(live & ~mover, ref, 0)
    ref = torch.cat([ref, ref.new_zeros(1)]).scatter(
        0, dst, torch.where(mover, st["book0"][B * MB:].long(), 0))[:NB]
    inside = (table >= 0) & (table < NB)
    table = torch.where(inside, to[torch.where(inside, table, 0)], table)
    used = (to.amax() + 1).view(1)
    return [table.to(I32), ref.to(I32), to.to(I32), used.to(I32), st["pools"][:, :, :NB]]


def _work_compact(c):
    each = max(1, min(c["MB"], int(c["NB"] * c["live"]) // c["B"]))
    live = min(c["NB"], each * c["B"])
    moved = live * (1 - live / c["NB"])
    page = 2 * c["L"] * c["Hkv"] * c["bs"] * c["D"] * 2
    return {"bytes": 2 * page * moved + 8 * c["B"] * c["MB"] + 12 * c["NB"], "flops": 0}


# ---------------------------------------------------------------------------

_OPS = {
    "append": (_prepare_append, _run_append, _work_append, _exact_append),
    "decode": (_prepare_decode, _run_decode, _work_decode, _exact_decode),
    "reserve": (_prepare_reserve, _run_reserve, _work_reserve, None),
    "fork": (_prepare_fork, _run_fork, _work_fork, None),
    "compact": (_prepare_compact, _run_compact, _work_compact, None),
}


def prepare(case, seed):
    return _OPS[case["op"]][0](case, torch.Generator(DEV).manual_seed(seed))


def run(state):
    return _OPS[state["c"]["op"]][1](state)


def work(case):
    return _OPS[case["op"]][2](case)


def exact(case, seed):
    f = _OPS[case["op"]][3]
    return None if f is None else f(case, seed)
