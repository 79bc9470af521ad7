"""GPU parity of the 4-bit cache: the append's rows byte for byte, their values, and decode
attention over ring, global and paged layers against float64.

Tolerance of the attention, per output o = sum_j w_j v_j over the stored values
v = c s + m (derived, with A = sum_j w_j (c s + |m|) and, per head, B the largest
sum_i |q_i| (c s + |m|) / sqrt(d) of a key):
  - scores: a group's products are accumulated in fp32 over two 16-term steps, scaled,
    and summed with the minimum's term: fewer than 24 roundings (2^-24; the tensor core
    may truncate: 2^-23) of partial sums that B bounds; exp2 adds 2^-22 relative.
    So a weight is off by eps = 24 * 2^-23 * B + 2^-21 relative, and o by 2 eps A;
  - the weights (times s) are rounded to fp16 before the second product: 2^-11 A for bf16
    calls; fp32 calls carry two fp16 parts: 2^-22 A;
  - the sums over keys in fp32, truncating at worst once per 16 keys: (n / 16) 2^-23 A;
  - the output's own rounding: half a step, 2^-8 |o| (bf16) or 2^-24 |o| (fp32).
The roundings are of either sign, so the root mean square error is far below the bound;
fp32 outputs are also held to an rms of 2e-5 (as the fp32 cache's elementwise bound).
"""
import numpy as np
import pytest
import torch

from oracle.sinkkv_oracle import clamp_sink_logits, kv4_pack, kv4_unpack, visible_positions

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sink_kv_attention_gb300 as m
    m._lib()
    return m


def f32(t):
    return t.detach().float().cpu().numpy()


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(shape, seed, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def rows_of(shape, D, seed, kscale=1.0, vscale=1.0):
    """Oracle-packed random rows [*shape, 5 D / 4] as a CUDA tensor."""
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((*shape, D)).astype(np.float32) * np.float32(kscale)
    v = rng.standard_normal((*shape, D)).astype(np.float32) * np.float32(vscale)
    return torch.from_numpy(kv4_pack(k, v)).cuda()


def attend64(q, rows, sink=None):
    """One sequence: q [Hq, D] float64, rows [Hkv, n, bytes] -> out, A [Hq, D], B [Hq] (see above)."""
    Hq, D = q.shape
    Hkv, n = rows.shape[:2]
    K, V = kv4_unpack(rows)
    mk, mv = _minima(rows)
    out, A, B = np.zeros((Hq, D)), np.zeros((Hq, D)), np.zeros(Hq)
    for h in range(Hq):
        g = h // (Hq // Hkv)
        s = K[g] @ q[h] / np.sqrt(D)
        z = -np.inf if sink is None else sink[h]
        m = max(s.max(), z)
        e = np.exp(s - m)
        w = e / (e.sum() + np.exp(z - m))
        out[h] = w @ V[g]
        A[h] = w @ (V[g] - mv[g] + np.abs(mv[g]))
        B[h] = ((K[g] - mk[g] + np.abs(mk[g])) @ np.abs(q[h])).max() / np.sqrt(D)
    return out, A, B


def _minima(rows):
    """The m of every value's group, [..., D] each for K and V."""
    D = rows.shape[-1] * 4 // 5
    out = []
    for o in (0, D // 2 + D // 8):
        p = np.ascontiguousarray(rows[..., o + D // 2:o + D // 2 + D // 8]).view("<u2")[..., 0::2]
        out.append((p.astype(np.uint32) << 16).view(np.float32).astype(np.float64).repeat(32, -1))
    return out


def check(got, want, A, B, n, dtype):
    half = torch.finfo(dtype).eps / 2
    eps = 24 * 2.0 ** -23 * B[:, None] + 2.0 ** -21
    p = 2.0 ** -11 if dtype == BF else 2.0 ** -22
    tol = half * np.abs(want) + (2 * eps + p + (n / 16 + 1) * 2.0 ** -23) * A * (1 + half) + 1e-30
    err = np.abs(got - want)
    assert np.all(err <= tol), (float((err / tol).max()), float(err.max()))
    if dtype == F32:
        assert np.sqrt((err ** 2).mean()) <= 2e-5 * max(1.0, float(A.max())), float(err.max())


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def _same_state(a, b):
    for f in ("pos", "head", "count"):
        x, y = getattr(a, f), getattr(b, f)
        assert (x is None and y is None) or torch.equal(x, y), f


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,r,neox", [(128, 128, True), (128, 64, False), (64, 64, True), (64, 32, False)])
@pytest.mark.parametrize("kind", ["ring", "global"])
def test_append_rows_are_the_oracles_bytes(sk, dtype, D, r, neox, kind):
    """Chunks of many lengths: q and k rotated to the same bits as for an unquantised cache,
    the same slots and state, and rows equal to the oracle's packing of what k and v hold;
    rows that no token went to keep their bytes."""
    B, Hq, Hkv, S, W = 3, 6, 3, 2, 11
    cap = 60
    table = sk.RopeTable(D, r, 1e4, 256, neox=neox)
    make = dict(sinks=S, window=W) if kind == "ring" else dict(capacity=cap)
    kd = sk.SK_LAYER_RING if kind == "ring" else sk.SK_LAYER_GLOBAL
    a = sk.KVLayer.allocate(kd, B, Hkv, D, bits=4, **make)
    ref = sk.KVLayer.allocate(kd, B, Hkv, D, k_dtype=dtype, v_dtype=dtype, **make)
    a.k.fill_(0xA5)
    start = torch.tensor([0, 1, 9], device="cuda")
    for L in (a, ref):
        L.pos.copy_(start)
        if kind == "ring":
            L.count.copy_((start - S).clamp(min=0).int())
            L.head.copy_(((start - S).clamp(min=0) % W).int())
    ref.k.fill_(7.0)   # a slot that no token reaches keeps its 7s
    ref.v.fill_(7.0)
    for i, T in enumerate([1, 1, 2, 5, 3, 11, 12, 14, 1]):
        q, k, v = randn((B, T, Hq, D), 10 + i, dtype), randn((B, T, Hkv, D), 30 + i, dtype), \
            randn((B, T, Hkv, D), 50 + i, dtype)
        q2, k2 = q.clone(), k.clone()
        sk.kv_append(table, a, q, k, v)
        sk.kv_append(table, ref, q2, k2, v.clone())
        assert torch.equal(q, q2) and torch.equal(k, k2)
        _same_state(a, ref)
        K, V = f32(ref.k), f32(ref.v)
        want = kv4_pack(K, V)
        blank = (K == 7.0).all(-1) & (V == 7.0).all(-1)
        want[blank] = 0xA5
        assert np.array_equal(a.k.cpu().numpy(), want), T
    assert a.error_bits() == 0


def test_append_of_rotated_keys_and_odd_heads(sk):
    """No table: keys as given; 5 kv heads, a batch of one, a value range over many decades."""
    D, Hkv, T = 128, 5, 37
    a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, 1, Hkv, D, capacity=T, bits=4)
    k = randn((1, T, Hkv, D), 1) * torch.logspace(-30, 30, T, device="cuda")[None, :, None, None]
    v = randn((1, T, Hkv, D), 2) * torch.logspace(30, -30, T, device="cuda")[None, :, None, None] + 3.0
    k[0, 3] = 0.0
    v[0, 4] = -1.5
    sk.kv_append(None, a, None, k.clone(), v)
    assert np.array_equal(a.k.cpu().numpy()[0], kv4_pack(f32(k[0]), f32(v[0])).transpose(1, 0, 2))


def test_append_refuses_on_the_device_as_other_caches_do(sk):
    D = 64
    a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, 2, 2, D, capacity=4, bits=4)
    a.k.fill_(9)
    a.pos.copy_(torch.tensor([3, 1]))
    k, v = randn((2, 2, 2, D), 1, BF), randn((2, 2, 2, D), 2, BF)
    sk.kv_append(None, a, None, k, v)
    assert a.error_bits() == sk.SK_DEVERR_CAPACITY and a.pos.tolist() == [3, 3]
    assert bool((a.k[0] == 9).all())
    assert np.array_equal(a.k[1, :, 1:3].cpu().numpy(), kv4_pack(f32(k[1]), f32(v[1])).transpose(1, 0, 2))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bs", [4, 16, 64])
def test_paged_append_rows(sk, dtype, bs):
    B, Hq, Hkv, D = 3, 4, 2, 128
    MB = -(-40 // bs) + 1
    P = sk.PagedLayer.allocate(B, Hkv, D, block_size=bs, n_blocks=B * MB + 2, max_blocks=MB, bits=4)
    ref = sk.PagedLayer.allocate(B, Hkv, D, block_size=bs, n_blocks=B * MB + 2, max_blocks=MB, dtype=dtype)
    perm = torch.randperm(B * MB, generator=torch.Generator().manual_seed(3)).int().view(B, MB).cuda()
    table = sk.RopeTable(D, D, 1e4, 128)
    P.k_pool.fill_(0x5A)
    ref.k_pool.fill_(7.0)
    ref.v_pool.fill_(7.0)
    for L in (P, ref):
        L.block_table.copy_(perm)
        L.seq_lens.copy_(torch.tensor([0, 3, 16]))
    for i, T in enumerate([1, 13, 7]):
        q, k, v = (randn((B, T, h, D), 10 * i + j, dtype) for j, h in enumerate((Hq, Hkv, Hkv)))
        sk.paged_append(table, ref, q.clone(), k.clone(), v)
        sk.paged_append(table, P, q, k, v)
        K, V = f32(ref.k_pool), f32(ref.v_pool)
        want = kv4_pack(K, V)
        want[(K == 7.0).all(-1) & (V == 7.0).all(-1)] = 0x5A
        assert np.array_equal(P.k_pool.cpu().numpy(), want)
    assert P.seq_lens.tolist() == ref.seq_lens.tolist() and P.error_bits() == 0


def test_non_finite_values_spoil_their_group_only(sk):
    D = 128
    a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, 1, 1, D, capacity=6, bits=4)
    k, v = randn((1, 6, 1, D), 1), randn((1, 6, 1, D), 2)
    clean = kv4_unpack(kv4_pack(f32(k), f32(v)))
    bad = [float("nan"), float("inf"), float("-inf")]
    for i, x in enumerate(bad):
        k[0, i, 0, 40] = x
        v[0, i, 0, 100] = x
    sk.kv_append(None, a, None, k, v)
    K, V = (t[0, 0].cpu().double().numpy() for t in sk.kv4_unpack(a.k, dtype=F32))
    for i in range(6):
        for got, want, grp in ((K, clean[0], 1), (V, clean[1], 3)):
            hit = np.arange(D) // 32 == grp
            if i < 3:
                assert not np.isfinite(got[i][hit]).any()
            else:
                hit[:] = False
            # fp32 values of code s + m: one rounding
            assert np.allclose(got[i][~hit], want[0, i, 0][~hit], rtol=2.0 ** -24, atol=0)


# ---------------------------------------------------------------------------
# unpack
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [0, 1, 3, 1000])
def test_unpack(sk, D, n):
    rng = np.random.default_rng(n)
    rows = rng.integers(0, 256, (n, D * 5 // 4), dtype=np.uint8)
    for o in (D // 2, D // 2 + D // 8 + D // 2):   # finite m and s >= 0
        p = rng.standard_normal((n, D // 16)).astype(np.float32)
        p[:, 1::2] = np.abs(p[:, 1::2])
        rows[:, o:o + D // 8] = (p.view(np.uint32) >> 16).astype("<u2").view(np.uint8)
    want = kv4_unpack(rows)
    dev = torch.from_numpy(rows).cuda()
    for dtype in (BF, F32):
        got = sk.kv4_unpack(dev, dtype=dtype)
        for x, y in zip(got, want):
            assert x.shape == (n, D) and x.dtype == dtype
            # the fp32 value, rounded once more for bf16
            z = torch.from_numpy(y).float().to(dtype)
            assert torch.equal(x.cpu(), z)


# ---------------------------------------------------------------------------
# decode attention
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rep", [1, 2, 4, 8])
def test_global_decode(sk, dtype, D, rep):
    """Lengths around the 32-row tile, zero among them, and one cut between many blocks."""
    lens = [0, 1, 2, 31, 32, 33, 64, 100, 997]
    B, Hkv = len(lens), 2
    cap = max(lens)
    rows = rows_of((B, Hkv, cap), D, 7)
    a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, B, Hkv, D, capacity=cap, bits=4)
    a.k.copy_(rows)
    for b, n in enumerate(lens):
        a.k[b, :, n:] = 0xFF      # rows that are not visible: NaN parameters
    a.pos.copy_(torch.tensor(lens))
    q = randn((B, Hkv * rep, D), 8, dtype)
    out = f64(sk.decode_attention(a, q))
    host = rows.cpu().numpy()
    for b, n in enumerate(lens):
        if n == 0:
            assert not out[b].any()
            continue
        want, A, Bs = attend64(f64(q[b]), host[b, :, :n])
        check(out[b], want, A, Bs, n, dtype)
    assert a.error_bits() == 0


@pytest.mark.parametrize("dtype,Hkv,rep", [(BF, 8, 4), (F32, 1, 8), (BF, 3, 1)])
def test_ring_decode(sk, dtype, Hkv, rep):
    """Rings that hold only sinks, part of the window, and all of it; learned sinks."""
    D, S, W = 128, 4, 500
    pos = [1, 4, 5, 300, 504, 505, 9000]
    B = len(pos)
    a = sk.KVLayer.allocate(sk.SK_LAYER_RING, B, Hkv, D, sinks=S, window=W, bits=4)
    rows = rows_of((B, Hkv, S + W), D, 11)
    a.k.copy_(rows)
    count = [min(W, max(0, p - S)) for p in pos]
    for b in range(B):
        a.k[b, :, min(pos[b], S) + count[b]:] = 0xFF
    a.pos.copy_(torch.tensor(pos))
    a.count.copy_(torch.tensor(count))
    a.head.copy_(torch.tensor([c % W for c in count]))
    q = randn((B, Hkv * rep, D), 12, dtype)
    for sink in (None, torch.linspace(-20, 20, Hkv * rep, device="cuda")):
        out = f64(sk.decode_attention(a, q, sink_logits=sink))
        z = None if sink is None else clamp_sink_logits(f64(sink))
        for b in range(B):
            n = min(pos[b], S) + count[b]
            want, A, Bs = attend64(f64(q[b]), rows[b, :, :n].cpu().numpy(), z)
            check(out[b], want, A, Bs, n, dtype)
    assert a.error_bits() == 0


@pytest.mark.parametrize("dtype,D,rep,bs,S,W,nsb", [
    (BF, 128, 4, 16, 4, 100, 0), (BF, 128, 8, 4, 2, 50, 2), (F32, 64, 2, 8, 0, 37, 0), (BF, 64, 1, 32, 0, 0, 1),
    (F32, 128, 4, 256, 3, 517, 1), (BF, 128, 2, 64, 70, 40, 0)])
def test_paged_decode(sk, dtype, D, rep, bs, S, W, nsb):
    """Pages in no order, blocks behind the window freed (-1), static sink blocks in front,
    lengths that end inside a page and a request of none."""
    lens = [0, 1, bs, bs + 1, 2 * bs + 3, 333, 1100]
    B, Hkv = len(lens), 2
    MB = -(-max(lens) // bs) + 2
    nb = B * MB + nsb
    P = sk.PagedLayer.allocate(B, Hkv, D, block_size=bs, n_blocks=nb, max_blocks=MB, sinks=S, window=W,
                               n_sink_blocks=nsb, bits=4)
    rows = rows_of((nb, Hkv, bs), D, 21)
    P.k_pool.copy_(rows)
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(5))
    table = perm[:B * MB].view(B, MB).int()
    sink_ids = perm[B * MB:].int()
    if nsb:
        P.sink_block_ids.copy_(sink_ids)
    P.seq_lens.copy_(torch.tensor(lens))
    host = rows.cpu().numpy()
    sink_len = nsb * bs
    q = randn((B, Hkv * rep, D), 22, dtype)
    want = []
    for b, n in enumerate(lens):
        if n == 0:
            want.append(None)
            continue
        L = n + sink_len
        vis = visible_positions(L - 1, S + W, S) if W > 0 else list(range(L))
        full = [int(sink_ids[i // bs]) if i < sink_len else int(table[b, (i - sink_len) // bs]) for i in range(L)]
        want.append(attend64(f64(q[b]), np.stack([host[full[i], :, i % bs] for i in vis], 1)) + (len(vis),))
        used = {(i - sink_len) // bs for i in vis if i >= sink_len}
        for j in range(MB):
            if j not in used:
                table[b, j] = -1
    P.block_table.copy_(table)
    out = f64(sk.paged_decode_attention(P, q))
    for b, w in enumerate(want):
        if w is None:
            assert not out[b].any()
        else:
            check(out[b], w[0], w[1], w[2], w[3], dtype)
    assert P.error_bits() == 0


def test_paged_decode_reports_a_bad_block(sk):
    P = sk.PagedLayer.allocate(1, 1, 64, block_size=16, n_blocks=4, max_blocks=3, bits=4)
    P.block_table.copy_(torch.tensor([[2, 4, 1]]))
    P.seq_lens.fill_(40)
    sk.paged_decode_attention(P, randn((1, 1, 64), 1, BF))
    assert P.error_bits() == sk.SK_DEVERR_BLOCK_TABLE


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("qs,ks,vs", [(1e4, 1.0, 1.0), (1e-20, 1.0, 1e-12), (1.0, 30.0, 1e12), (3e37, 1e-37, 1.0),
                                      (1e-30, 1e30, 1.0)])
def test_magnitudes(sk, dtype, qs, ks, vs):
    """q, K and V far from 1: the references and the fp16 operands follow their ranges."""
    if qs > 1e34:
        qs, ks = 1e33, 1e-33      # |q| < 2^116
    D, n, Hq, Hkv = 128, 200, 8, 2
    rows = rows_of((1, Hkv, n), D, 31, ks, vs)
    a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, 1, Hkv, D, capacity=n, bits=4)
    a.k.copy_(rows)
    a.pos.fill_(n)
    q = (randn((1, Hq, D), 32) * qs).to(dtype)
    out = f64(sk.decode_attention(a, q))[0]
    want, A, Bs = attend64(f64(q[0]), rows[0].cpu().numpy())
    half = torch.finfo(dtype).eps / 2
    eps = 24 * 2.0 ** -23 * Bs[:, None] + 2.0 ** -21
    tol = half * np.abs(want) + (2 * np.expm1(np.minimum(eps, 10)) + (2.0 ** -11 if dtype == BF else 2.0 ** -22) +
                                 14 * 2.0 ** -23) * A * (1 + half)
    assert np.all(np.abs(out - want) <= tol)


def test_scales_over_many_decades_within_one_sequence(sk):
    """V scales that grow along the keys move the reference again and again, and keys whose
    values are tiny beside the largest keep their weight in the sum of weights."""
    D, n = 128, 640
    rng = np.random.default_rng(41)
    k = rng.standard_normal((1, 1, n, D)).astype(np.float32)
    mag = np.exp2(np.linspace(-40, 20, n)).astype(np.float32)
    for order in (1, -1):
        v = rng.standard_normal((1, 1, n, D)).astype(np.float32) * mag[::order, None]
        rows = kv4_pack(k, v)
        a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, 1, 1, D, capacity=n, bits=4)
        a.k.copy_(torch.from_numpy(rows))
        a.pos.fill_(n)
        q = randn((1, 4, D), 42)
        out = f64(sk.decode_attention(a, q))[0]
        want, A, Bs = attend64(f64(q[0]), rows[0])
        check(out, want, A, Bs, n, F32)


def test_non_finite_groups_stay_where_they_are(sk):
    """An infinite V spoils its group of dims and leaves the others; a NaN key spoils its kv
    head's outputs and leaves the other head's."""
    D, n = 128, 70
    k, v = randn((1, n, 2, D), 51), randn((1, n, 2, D), 52)
    a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, 1, 2, D, capacity=n, bits=4)
    b = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, 1, 2, D, capacity=n, bits=4)
    sk.kv_append(None, b, None, k.clone(), v)
    v2, k2 = v.clone(), k.clone()
    v2[0, 33, 0, 70] = float("inf")
    k2[0, 5, 1, 3] = float("nan")
    sk.kv_append(None, a, None, k2, v2)
    q = randn((1, 4, D), 53, BF)
    x, y = sk.decode_attention(a, q)[0], sk.decode_attention(b, q)[0]
    hit = torch.arange(D, device="cuda") // 32 == 2
    assert not torch.isfinite(x[:2][:, hit]).any()
    assert torch.equal(x[:2][:, ~hit], y[:2][:, ~hit])
    assert torch.isnan(x[2:]).all()


def test_rows_past_4_gib(sk):
    """Row offsets past 2^32 bytes: the last kv head of a 4.4 GB cache, mostly zero rows."""
    D, Hkv, n = 128, 8, 3_450_000
    a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, 1, Hkv, D, capacity=n, bits=4)
    assert a.k.numel() > 1 << 32
    one = kv4_pack(np.zeros(D, np.float32), np.ones(D, np.float32))
    m = 150_000
    for g in range(Hkv):      # the last m (g + 1) / 8 rows hold ones, the others zeros
        a.k[0, g, n - m * (g + 1) // 8:] = torch.from_numpy(one).cuda()
    a.pos.fill_(n)
    out = f64(sk.decode_attention(a, randn((1, Hkv, D), 61)))[0]
    want = np.array([m * (g + 1) // 8 / n for g in range(Hkv)])[:, None]
    # sums of up to n equal fp32 terms, a lane's share of a warp's share: n / (152 * 12 * 8) of them in turn
    assert np.all(np.abs(out - want) <= want * (n / (152 * 12 * 8) * 2.0 ** -24 + 2.0 ** -20))


@pytest.mark.parametrize("dtype,rep", [(F32, 1), (BF, 1), (BF, 4)])
def test_a_full_batch_stays_inside_its_workspace(sk, dtype, rep):
    """1024 sequences of 32 kv heads: the workspace's last slots are used, and nothing behind
    it; heads far apart agree with float64."""
    D, B, Hkv, n = 64, 1024, 32, 37
    a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, B, Hkv, D, capacity=n, bits=4)
    rows = rows_of((3, Hkv, n), D, 75)
    a.k.copy_(rows.repeat(B // 3 + 1, 1, 1, 1)[:B])
    a.pos.copy_(torch.arange(B) * 7 % (n + 1))
    q = randn((B, Hkv * rep, D), 76, dtype)
    need = sk.decode_workspace_bytes(a, Hkv * rep)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    out = f64(sk.decode_attention(a, q, workspace=ws[:need]))
    assert (ws[need:] == 0x5A).all()
    for b in (0, 1, 500, 1022, 1023):
        m = b * 7 % (n + 1)
        if m == 0:
            assert not out[b].any()
            continue
        want, A, Bs = attend64(f64(q[b]), rows[b % 3, :, :m].cpu().numpy())
        check(out[b], want, A, Bs, m, dtype)


def test_a_length_past_the_block_table_is_reported(sk):
    """More tokens than the table has entries for: the error word says so, and every read
    stays inside the pool."""
    P = sk.PagedLayer.allocate(2, 2, 64, block_size=16, n_blocks=8, max_blocks=3, sinks=2, window=20, bits=4)
    P.block_table.copy_(torch.arange(6).view(2, 3))
    P.k_pool.copy_(rows_of((8, 2, 16), 64, 77))
    P.seq_lens.copy_(torch.tensor([1 << 60, 30]))
    q = randn((2, 4, 64), 78, BF)
    out = sk.paged_decode_attention(P, q)
    assert P.error_bits() == sk.SK_DEVERR_BLOCK_TABLE
    P.err.zero_()
    P.seq_lens.copy_(torch.tensor([48, 30]))
    again = sk.paged_decode_attention(P, q)
    assert torch.equal(out[1], again[1]) and P.error_bits() == 0


def test_rerotation_and_shift_refuse_4_bit_layers(sk):
    a = sk.KVLayer.allocate(sk.SK_LAYER_RING, 1, 2, 64, sinks=1, window=7, bits=4)
    t = [sk.RopeTable(64, 64, 1e4, 64, yarn_factor=f, yarn_orig_ctx=8) for f in (1.0, 2.0)]
    for call in (lambda: sk.kv_rerotate([a], t[0], t[1]), lambda: sk.kv_shift_recent([a], t[0], -1)):
        with pytest.raises(sk.SinkKVError) as e:
            call()
        assert e.value.status == sk.SK_ERR_UNSUPPORTED


def test_noalloc_and_given_buffers(sk):
    D, n, Hq, Hkv = 128, 300, 8, 2
    a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, 2, Hkv, D, capacity=n, bits=4)
    a.k.copy_(rows_of((2, Hkv, n), D, 71))
    a.pos.copy_(torch.tensor([n, 123]))
    q = randn((2, Hq, D), 72, BF)
    want = sk.decode_attention(a, q)
    out = torch.empty_like(q)
    sk.decode_attention_noalloc(a, q, out)
    assert torch.equal(out, want)
    ws = torch.full((sk.decode_workspace_bytes(a, Hq),), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(sk.decode_attention(a, q, workspace=ws), want)   # NaN left in the workspace
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = sk.decode_attention(a, q)
    side.synchronize()
    assert torch.equal(got, want)


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------

def test_steps_in_a_graph_equal_eager_steps(sk):
    D, Hq, Hkv, B, S, W = 128, 8, 2, 4, 2, 40
    table = sk.RopeTable(D, D, 1e4, 256)

    def fresh():
        return sk.KVLayer.allocate(sk.SK_LAYER_RING, B, Hkv, D, sinks=S, window=W, bits=4)

    steps = 50
    qs, ks, vs = (randn((steps, B, 1, h, D), 80 + h, BF) for h in (Hq, Hkv, Hkv + 1))
    vs = vs[:, :, :, :Hkv].contiguous()
    a, b = fresh(), fresh()
    want = []
    for i in range(steps):
        q = qs[i].clone()
        sk.kv_append(table, a, q, ks[i].clone(), vs[i])
        want.append(sk.decode_attention(a, q[:, 0].contiguous()))
    q, k, v = qs[0].clone(), ks[0].clone(), vs[0].clone()
    out = torch.empty(B, Hq, D, dtype=BF, device="cuda")
    ws = torch.empty(sk.decode_workspace_bytes(b, Hq), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sk.kv_append(table, b, q, k, v)
        sk.decode_attention(b, q[:, 0], out=out, workspace=ws)
    for i in range(steps):
        q.copy_(qs[i])
        k.copy_(ks[i])
        v.copy_(vs[i])
        g.replay()
        assert torch.equal(out, want[i]), i
    assert torch.equal(a.k, b.k)
    _same_state(a, b)


def test_units_cut_between_blocks_in_graphs_that_share_a_workspace(sk):
    """Sequences long enough to be cut between blocks: two captured calls of other shapes over
    one workspace, replayed in turn, and eager calls between them, always give the first
    call's bits (what a call leaves in the workspace never matters to the next)."""
    D = 128
    shapes = [(1, 2, 4, 20_000), (3, 3, 8, 7_001)]
    layers, qs, outs, graphs, want = [], [], [], [], []
    ws = torch.full((8 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    for i, (B, Hkv, rep, n) in enumerate(shapes):
        a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, B, Hkv, D, capacity=n, bits=4)
        sk.kv_append(None, a, None, randn((B, n, Hkv, D), 200 + i, BF), randn((B, n, Hkv, D), 210 + i, BF))
        a.pos.copy_(torch.tensor([n, n - 13, 5][:B]))
        layers.append(a)
        qs.append(randn((B, Hkv * rep, D), 220 + i, BF))
        outs.append(torch.zeros_like(qs[-1]))
        assert ws.numel() >= sk.decode_workspace_bytes(a, Hkv * rep)
        want.append(sk.decode_attention(a, qs[i], workspace=ws).clone())
        ref, A, Bs = attend64(f64(qs[i][0]), a.k[0].cpu().numpy())
        check(f64(want[i][0]), ref, A, Bs, n, BF)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sk.decode_attention(a, qs[i], out=outs[i], workspace=ws)
        graphs.append(g)
    for r in range(20):
        for i in (0, 1) if r % 3 else (1, 0, 0):
            outs[i].zero_()
            graphs[i].replay()
            assert torch.equal(outs[i], want[i]), (r, i)
        if r % 5 == 4:
            ws.random_(0, 256)
            assert torch.equal(sk.decode_attention(layers[1], qs[1], workspace=ws), want[1])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_two_calls_at_once(sk, dtype):
    """Calls of two streams that share the GPU, each with its own workspace, over units cut
    between blocks: always the bits of the call alone."""
    D, rep, cases = 128, 4, [(2, 2, 9001), (5, 4, 1500)]
    layers, qs, wss, want = [], [], [], []
    for i, (B, Hkv, n) in enumerate(cases):
        a = sk.KVLayer.allocate(sk.SK_LAYER_GLOBAL, B, Hkv, D, capacity=n, bits=4)
        a.k.copy_(rows_of((B, Hkv, n), D, 300 + i))
        a.pos.copy_(torch.tensor([n, n // 3, 0, 1, n - 1][:B]))
        layers.append(a)
        qs.append(randn((B, Hkv * rep, D), 310 + i, dtype))
        wss.append(torch.empty(sk.decode_workspace_bytes(a, Hkv * rep), dtype=torch.uint8, device="cuda"))
        want.append(sk.decode_attention(a, qs[i], workspace=wss[i]).clone())
    rounds = 40
    outs = [torch.zeros((rounds,) + tuple(q.shape), dtype=dtype, device="cuda") for q in qs]
    streams = [torch.cuda.Stream() for _ in cases]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for r in range(rounds):
        for i, st in enumerate(streams):
            sk.decode_attention(layers[i], qs[i], out=outs[i][r], workspace=wss[i], stream=st)
    torch.cuda.synchronize()
    for i in range(len(cases)):
        assert all(torch.equal(outs[i][r], want[i]) for r in range(rounds))


@pytest.mark.parametrize("kind", ["ring", "global"])
def test_prefill_over_a_4_bit_prior(sk, kind):
    """A chunk over a 4-bit prior gives the bits of the same chunk over a bf16 cache that
    holds the prior's values, and appends to it as any chunk does."""
    D, Hq, Hkv, B, S, W = 128, 8, 2, 2, 4, 150
    T0, T = 333, 130
    make = dict(sinks=S, window=W) if kind == "ring" else dict(capacity=T0 + T)
    kd = sk.SK_LAYER_RING if kind == "ring" else sk.SK_LAYER_GLOBAL
    a = sk.KVLayer.allocate(kd, B, Hkv, D, bits=4, **make)
    k0, v0 = randn((B, T0, Hkv, D), 91, BF), randn((B, T0, Hkv, D), 92, BF)
    sk.kv_append(None, a, None, k0, v0)
    K, V = sk.kv4_unpack(a.k)
    b = sk.KVLayer(kd, K, V, a.pos.clone(), a.sinks, a.window, None if a.head is None else a.head.clone(),
                   None if a.count is None else a.count.clone(), None, torch.zeros_like(a.err))
    q, k, v = (randn((B, T, h, D), 93 + i, BF) for i, h in enumerate((Hq, Hkv, Hkv)))
    s, w = (S, W) if kind == "ring" else (0, 0)
    x = sk.prefill_attention(q, k, v, T0, s, w, prior=a, err=a.err)
    y = sk.prefill_attention(q, k, v, T0, s, w, prior=b, err=b.err)
    assert torch.equal(x, y) and a.error_bits() == 0 and b.error_bits() == 0
    sk.kv_append(None, a, None, k, v)
    assert a.pos.tolist() == [T0 + T] * B


def test_a_prompt_and_its_decode_steps_stay_near_the_unquantised_cache(sk):
    """A prompt in two chunks, then decode steps: the 4-bit path end to end against the bf16
    path.  Each value is off by at most s / 2, so an output differs by at most the largest
    s / 2 of V plus what the keys' s / 2 do to the weights: with |dscore| <= sum_i |q_i| s_K / 2
    / sqrt(d) =: d for every key, weights move by a factor of at most e^(2 d)."""
    D, Hq, Hkv, B, S, W = 128, 8, 2, 2, 4, 200
    table = sk.RopeTable(D, D, 1e4, 1024)
    layers = [sk.KVLayer.allocate(sk.SK_LAYER_RING, B, Hkv, D, sinks=S, window=W, bits=bits) for bits in (4, None)]
    x = {h: randn((B, 400, h, D), 100 + h, BF) for h in (Hq, Hkv)}
    vals = randn((B, 400, Hkv, D), 110, BF)
    for lo, hi in ((0, 150), (150, 390)):
        for L in layers:
            q, k, v = x[Hq][:, lo:hi].clone(), x[Hkv][:, lo:hi].clone(), vals[:, lo:hi].contiguous()
            pos = torch.arange(lo, hi, device="cuda").repeat(B)
            sk.rope_apply(table, q.view(-1, Hq, D), pos)
            sk.rope_apply(table, k.view(-1, Hkv, D), pos)
            out = sk.prefill_attention(q, k, v, lo, S, W, prior=L if lo else None, err=L.err)
            assert torch.isfinite(out).all()
            sk.kv_append(None, L, None, k, v)
    for t in range(390, 400):
        got = []
        for L in layers:
            q, k, v = (y[:, t:t + 1].clone() for y in (x[Hq], x[Hkv], vals))
            sk.kv_append(table, L, q, k, v)
            got.append(f64(sk.decode_attention(L, q[:, 0].contiguous())))
        rows = layers[0].k.cpu().numpy()
        par = np.ascontiguousarray(rows[..., 64:80]).view("<u2")[..., 1::2], \
            np.ascontiguousarray(rows[..., 144:160]).view("<u2")[..., 1::2]
        s_k, s_v = ((p.astype(np.uint32) << 16).view(np.float32) for p in par)
        d = np.abs(f64(q[:, 0])).reshape(B, Hkv, 4, D).sum(-1).max(-1)[..., None] * s_k.max((-1, -2))[..., None]
        d = d.max() / 2 / np.sqrt(D)
        vmax = np.abs(f64(layers[1].v)).max()
        bound = s_v.max() / 2 + vmax * np.expm1(2 * d) + 2.0 ** -7 * vmax
        assert np.abs(got[0] - got[1]).max() <= bound
        # ... and in the mean far less: the steps' roundings are of either sign
        assert np.sqrt(((got[0] - got[1]) ** 2).mean()) <= s_v.max() / 2
    assert all(L.error_bits() == 0 for L in layers)
