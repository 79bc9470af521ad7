"""GPU parity of the page operations: tables, counts and pools against the oracle, which serves
one request after the other; then serving loops that reserve, append, attend, fork and
compact, against caches whose pages are never shared or moved."""
import numpy as np
import pytest
import torch

from oracle.sinkkv_oracle import pages_compact, pages_fork, pages_reserve

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sink_kv_attention_gb300 as m
    m._lib()
    return m


def build(sk, rng, B, MB, NB, bs, *, S=0, W=0, nsb=0, kinds=("bf16",), share=1, fill=0.5):
    """Layers over one table in a random state: runs of `share` rows hold the same pages, some
    pages are held by the caller; pools of random bits."""
    layers = []
    for kind in kinds:
        how = dict(bits=4) if kind == "i4" else dict(dtype=torch.float32 if kind == "f32" else torch.bfloat16)
        layers.append(sk.PagedLayer.allocate(B, 2, 64, block_size=bs, n_blocks=NB, max_blocks=MB, sinks=S, window=W,
                                             n_sink_blocks=nsb, **how))
    for x in layers[1:]:
        x.block_table, x.sink_block_ids, x.err = layers[0].block_table, layers[0].sink_block_ids, layers[0].err
    for x in layers:
        for pool in (x.k_pool, x.v_pool):
            if pool is not None:
                pool.view(torch.uint8).copy_(torch.from_numpy(
                    rng.integers(0, 120, pool.view(torch.uint8).shape, dtype=np.uint8)))
    perm = rng.permutation(NB)
    sink_ids, perm = perm[:nsb], perm[nsb:]
    ref = np.zeros(NB, np.int64)
    ref[sink_ids] = 1
    held, perm = perm[:NB // 16], perm[NB // 16:]
    ref[held] = 1
    table = np.full((B, MB), -1)
    lens = np.zeros(B, np.int64)
    for b in range(0, B, share):
        n = min(int(rng.integers(0, max(1, int(fill * MB)) + 1)), len(perm))
        rows = range(b, min(B, b + share))
        pages, perm = perm[:n], perm[n:]
        for r in rows:
            table[r, :n] = pages
            ref[pages] += 1
            lens[r] = max(0, n * bs - int(rng.integers(0, bs)))
        if share > 1 and rng.random() < 0.7:
            lens[list(rows)] = lens[b]
    for x in layers:
        x.block_table.copy_(torch.from_numpy(table))
        x.seq_lens.copy_(torch.from_numpy(lens))
        if nsb:
            x.sink_block_ids.copy_(torch.from_numpy(sink_ids.copy()))
    group = sk.PagedGroup(layers, ref=torch.from_numpy(ref).int().cuda())
    return layers, group, table, ref, lens, sink_ids


def pools_of(layers):
    return [p.view(torch.uint8).cpu().numpy().copy() for x in layers for p in (x.k_pool, x.v_pool) if p is not None]


def check_state(layers, group, table, ref, pools=None):
    assert np.array_equal(layers[0].block_table.cpu().numpy(), table)
    assert np.array_equal(group.ref.cpu().numpy(), ref)
    if pools is not None:
        for got, want in zip(pools_of(layers), pools):
            assert np.array_equal(got, want)


RESERVE = [  # B, MB, NB, bs, S, W, nsb, share, fill, most new tokens, kinds
    (1, 4, 8, 4, 0, 0, 0, 1, 0.5, 3, ("bf16",)),
    (5, 9, 64, 8, 0, 0, 0, 1, 0.7, 40, ("bf16", "f32", "i4")),
    (12, 16, 200, 16, 0, 0, 0, 4, 0.8, 1, ("i4", "bf16")),
    (12, 16, 80, 16, 0, 0, 0, 4, 0.8, 60, ("bf16",)),             # the pool runs out
    (40, 33, 1000, 4, 3, 21, 0, 3, 0.9, 9, ("f32",)),             # window and sinks
    (40, 33, 900, 16, 40, 100, 2, 2, 0.9, 30, ("i4",)),           # static sink blocks in front
    (300, 70, 9000, 16, 0, 0, 0, 1, 0.5, 300, ("bf16",)),         # more requests than warps
    (1024, 12, 20000, 16, 0, 50, 0, 8, 0.9, 20, ("bf16",)),
]


@pytest.mark.parametrize("case", RESERVE, ids=[f"case{i}" for i in range(len(RESERVE))])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_reserve(sk, case, seed):
    B, MB, NB, bs, S, W, nsb, share, fill, most, kinds = case
    rng = np.random.default_rng(100 * seed + B)
    layers, group, table, ref, lens, _ = build(sk, rng, B, MB, NB, bs, S=S, W=W, nsb=nsb, kinds=kinds, share=share,
                                               fill=fill)
    pools = pools_of(layers)
    n_new = rng.integers(0, most + 1, B)
    if seed == 2:
        n_new[rng.integers(0, B)] = MB * bs + 1        # passes the table: refused alone
        n_new[:] = np.where(n_new == 0, -3, n_new)
    granted = group.reserve(torch.from_numpy(n_new).int().cuda())
    want, copies = pages_reserve(table, ref, lens.tolist(), n_new.tolist(), bs, S, W, nsb * bs)
    for src, dst in copies:
        for p in pools:
            p[dst] = p[src]
    assert granted.tolist() == want
    check_state(layers, group, table, ref, pools)
    bits = layers[0].error_bits()
    assert bool(bits & sk.SK_DEVERR_CAPACITY) == (0 in want) and not bits & ~sk.SK_DEVERR_CAPACITY
    assert np.array_equal(layers[0].seq_lens.cpu().numpy(), lens)
    # asked again, nothing changes: every block is there and held alone
    layers[0].err.zero_()
    again = group.reserve(torch.from_numpy(np.where(np.array(want) == 1, n_new, 0)).int().cuda())
    assert again.tolist() == [1] * B
    check_state(layers, group, table, ref, pools)


def test_reserve_one_token_by_default_and_refusals(sk):
    rng = np.random.default_rng(7)
    layers, group, table, ref, lens, _ = build(sk, rng, 6, 5, 40, 8, fill=0.8)
    lens[:] = [0, 8, 3, 40, -1, 11]
    table[2, 0] = 1000                                     # a partly filled block outside the pool
    table[5, 1] = -1                                       # ... and one that is missing
    layers[0].seq_lens.copy_(torch.from_numpy(lens))
    layers[0].block_table.copy_(torch.from_numpy(table))
    granted = group.reserve()
    want, _ = pages_reserve(table, ref, lens.tolist(), [1] * 6, 8, 0, 0, 0)
    assert granted.tolist() == want == [1, 1, 0, 0, 0, 0]
    check_state(layers, group, table, ref)
    assert layers[0].error_bits() == sk.SK_DEVERR_CAPACITY | sk.SK_DEVERR_BLOCK_TABLE | sk.SK_DEVERR_STATE


@pytest.mark.parametrize("B,MB,NB", [(1, 1, 4), (4, 7, 40), (33, 20, 300), (256, 130, 9000), (1024, 9, 4000)])
def test_fork(sk, B, MB, NB):
    rng = np.random.default_rng(B)
    layers, group, table, ref, lens, _ = build(sk, rng, B, MB, NB, 8, kinds=("bf16", "i4", "bf16"), share=2, fill=0.9)
    layers[2].seq_lens = layers[0].seq_lens                # two layers share their lengths
    layers[1].seq_lens.add_(1)
    group = sk.PagedGroup(layers, ref=group.ref)
    both = np.stack([lens, lens + 1])
    for step in range(3):
        parents = rng.integers(-1, B, B)
        parents[rng.random(B) < 0.3] = -1
        stay = rng.random(B) < 0.3
        parents[stay] = np.arange(B)[stay]
        group.fork(torch.from_numpy(parents).int().cuda())
        pages_fork(table, ref, both, parents)
        check_state(layers, group, table, ref)
        assert np.array_equal(layers[0].seq_lens.cpu().numpy(), both[0])
        assert np.array_equal(layers[1].seq_lens.cpu().numpy(), both[1])
    assert layers[0].error_bits() == 0


def test_fork_reports_a_bad_parent(sk):
    rng = np.random.default_rng(3)
    layers, group, table, ref, lens, _ = build(sk, rng, 4, 6, 40, 8, fill=0.9)
    parents = np.array([4, 0, -2, 1])
    group.fork(torch.from_numpy(parents).int().cuda())
    both = lens[None].copy()
    pages_fork(table, ref, both, parents)
    check_state(layers, group, table, ref)
    assert layers[0].seq_lens.tolist() == both[0].tolist() and layers[0].error_bits() == sk.SK_DEVERR_STATE


@pytest.mark.parametrize("B,MB,NB,nsb,share,kinds", [
    (1, 1, 5, 0, 1, ("bf16",)), (3, 5, 33, 0, 2, ("i4", "f32")), (20, 9, 257, 3, 1, ("bf16",)),
    (64, 40, 5000, 0, 1, ("i4",)), (64, 60, 4100, 7, 2, ("bf16", "i4")), (9, 3, 60000, 1, 1, ("i4",))])
def test_compact(sk, B, MB, NB, nsb, share, kinds):
    rng = np.random.default_rng(NB)
    layers, group, table, ref, lens, sink_ids = build(sk, rng, B, MB, NB, 8, nsb=nsb, kinds=kinds, share=share,
                                                      fill=0.9)
    table[0, -1] = NB + 3                                  # outside the pool: left as it is
    layers[0].block_table.copy_(torch.from_numpy(table))
    pools = pools_of(layers)
    block_map, used = group.compact()
    want_map, want_used, moves = pages_compact(table, ref, sink_ids)
    for src, dst in moves:
        for p in pools:
            p[dst] = p[src]
    assert np.array_equal(block_map.cpu().numpy(), want_map) and used.item() == want_used
    check_state(layers, group, table, ref, pools)
    block_map, used = group.compact()                      # nothing is left to move
    assert np.array_equal(block_map.cpu().numpy(), np.where(ref > 0, np.arange(NB), -1))
    assert used.item() == want_used
    check_state(layers, group, table, ref, pools)
    assert layers[0].error_bits() == 0


@pytest.mark.parametrize("B,n_layers", [(4, 3), (6, 41), (200, 31), (2, 128)])
def test_copies_and_moves_in_many_layers_of_unequal_pages(sk, B, n_layers):
    """A reserve that copies half of the requests' last pages, then a compaction, in pools whose
    pages differ in size (pieces of a page that a smaller one has not are not moved)."""
    rng = np.random.default_rng(B + n_layers)
    kinds = [("i4", "bf16", "f32")[int(rng.integers(0, 3))] for _ in range(n_layers)]
    layers, group, table, ref, lens, sink_ids = build(sk, rng, B, 5, 6 * B + 8, 32, kinds=kinds, share=2, fill=0.9)
    pools = pools_of(layers)
    granted = group.reserve()
    want, copies = pages_reserve(table, ref, lens.tolist(), [1] * B, 32, 0, 0, 0)
    for src, dst in copies:
        for p in pools:
            p[dst] = p[src]
    assert granted.tolist() == want
    check_state(layers, group, table, ref, pools)
    block_map, used = group.compact()
    want_map, want_used, moves = pages_compact(table, ref, sink_ids)
    for src, dst in moves:
        for p in pools:
            p[dst] = p[src]
    assert np.array_equal(block_map.cpu().numpy(), want_map) and used.item() == want_used
    check_state(layers, group, table, ref, pools)


def test_compact_of_an_empty_pool(sk):
    P = sk.PagedLayer.allocate(2, 2, 64, block_size=8, n_blocks=100, max_blocks=3)
    block_map, used = sk.PagedGroup([P]).compact()
    assert used.item() == 0 and (block_map == -1).all()


def test_pages_past_4_gib(sk):
    """A copy and a move between pages whose byte offsets pass 2^32."""
    NB, bs = 70_000, 128                                   # 64 KB a page: 4.6 GB
    P = sk.PagedLayer(torch.zeros(NB, 2, bs, 128, dtype=torch.bfloat16, device="cuda"),
                      torch.zeros(NB, 2, bs, 128, dtype=torch.bfloat16, device="cuda"),
                      torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), None,
                      torch.tensor([5, 5], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), 0, 0)
    ref = torch.ones(NB, dtype=torch.int32, device="cuda")
    a, b = NB - 3, NB - 1
    P.block_table[:, 0] = a
    ref[a], ref[b] = 2, 0
    x = torch.randn(2, bs, 128, device="cuda").bfloat16()
    P.k_pool[a], P.v_pool[a] = x, -x
    g = sk.PagedGroup([P], ref=ref)
    assert g.reserve().tolist() == [1, 1]
    assert P.block_table[:, 0].tolist() == [b, a] and torch.equal(P.k_pool[b], x) and torch.equal(P.v_pool[b], -x)
    ref[7] = 0
    block_map, used = g.compact()
    assert block_map[b].item() == 7 and used.item() == NB - 1 and P.block_table[0, 0].item() == 7
    assert torch.equal(P.k_pool[7], x) and torch.equal(P.v_pool[7], -x)


@pytest.mark.parametrize("bits", [None, 4])
def test_beams_decode_as_if_their_pages_were_their_own(sk, bits):
    """Two requests of three beams each: prompts appended once and forked, then steps that
    reserve, append, attend and reorder, with a compaction in between; next to it the same
    tokens in caches without sharing, whose rows are copied whole at each reorder."""
    B, Hq, Hkv, D, bs, MB, NB, layers_n = 6, 8, 2, 128, 16, 12, 60, 2
    how = dict(bits=4) if bits else {}
    gen = torch.Generator().manual_seed(9)

    def rand(T, H):
        return torch.randn(B, T, H, D, generator=gen).bfloat16().cuda()

    table = sk.RopeTable(D, D, 1e4, 256)
    mine = [sk.PagedLayer.allocate(B, Hkv, D, block_size=bs, n_blocks=NB, max_blocks=MB, **how) for _ in range(layers_n)]
    for x in mine[1:]:
        x.block_table, x.err = mine[0].block_table, mine[0].err
    group = sk.PagedGroup(mine)
    own = [sk.PagedLayer.allocate(B, Hkv, D, block_size=bs, n_blocks=B * MB, max_blocks=MB, **how)
           for _ in range(layers_n)]
    for x in own:
        x.block_table.copy_(torch.arange(B * MB).view(B, MB))

    def own_fork(parents):
        for x in own:
            rows = torch.where(parents < 0, 0, parents).long()
            for pool in (x.k_pool, x.v_pool):
                if pool is not None:
                    y = pool.view(B, MB, *pool.shape[1:])
                    y.copy_(y[rows])
            x.seq_lens.copy_(torch.where(parents < 0, 0, x.seq_lens[rows]))

    def step(T, rows):
        """T tokens for the rows given (the others append nothing)."""
        n_new = torch.zeros(B, dtype=torch.int32, device="cuda")
        n_new[rows] = T
        assert group.reserve(n_new).tolist() == [1] * B
        sub = torch.tensor(rows, device="cuda")
        outs = []
        for i in range(layers_n):
            q, k, v = rand(T, Hq)[sub], rand(T, Hkv)[sub], rand(T, Hkv)[sub]
            for x, keep in ((mine[i], outs), (own[i], outs)):
                part = sk.PagedLayer(x.k_pool, x.v_pool, x.block_table[sub].contiguous(), None,
                                     x.seq_lens[sub].contiguous(), x.err, 0, 0)
                qq = q.clone()
                sk.paged_append(table, part, qq, k.clone(), v)
                x.seq_lens[sub] = part.seq_lens
                keep.append(sk.paged_decode_attention(part, qq[:, -1].contiguous()))
        for i in range(0, len(outs), 2):
            assert torch.equal(outs[i], outs[i + 1])

    step(37, [0])
    step(21, [3])
    first = torch.tensor([0, 0, 0, 3, 3, 3], dtype=torch.int32, device="cuda")
    group.fork(first)
    own_fork(first)
    assert group.ref.max().item() == 3
    for t in range(40):
        step(1, list(range(B)))
        if t % 3 == 1:
            r = torch.randint(0, 3, (B,), generator=gen)
            parents = (torch.arange(B) // 3 * 3 + r).int().cuda()
            group.fork(parents)
            own_fork(parents)
        if t == 20:
            _, used = group.compact()
            assert used.item() == (group.ref > 0).sum().item()
    gone = torch.tensor([-1, 1, -1, -1, -1, -1], dtype=torch.int32, device="cuda")
    group.fork(gone)
    own_fork(gone)
    step(3, [1])
    tab = mine[0].block_table.cpu().numpy()
    assert np.array_equal(group.ref.cpu().numpy(), np.bincount(tab[tab >= 0].ravel(), minlength=NB))
    assert mine[0].error_bits() == 0 and own[0].error_bits() == 0


def test_a_window_gives_its_pages_back_in_a_graph(sk):
    """A captured step of reserve, append and attention over a 4-bit windowed layer: the pool
    never needs more than the window's pages, however long the requests grow."""
    B, Hq, Hkv, D, bs, S, W = 3, 4, 1, 64, 4, 2, 19
    per = 1 + (W + bs - 1) // bs + 1                       # sink page, window pages, one more
    P = sk.PagedLayer.allocate(B, Hkv, D, block_size=bs, n_blocks=B * per, max_blocks=64, sinks=S, window=W, bits=4)
    ring = sk.KVLayer.allocate(sk.SK_LAYER_RING, B, Hkv, D, sinks=S, window=W, bits=4)
    g = sk.PagedGroup([P])
    table = sk.RopeTable(D, D, 1e4, 256)
    q, k, v = (torch.zeros(B, 1, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    granted = torch.zeros(B, dtype=torch.int32, device="cuda")
    out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(sk.paged_decode_workspace_bytes(P, Hq), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.reserve(granted=granted)
        sk.paged_append(table, P, q, k, v)
        sk.paged_decode_attention(P, q[:, 0], out=out, workspace=ws)
    gen = torch.Generator().manual_seed(4)
    for t in range(200):
        x = [torch.randn(B, 1, h, D, generator=gen).bfloat16().cuda() for h in (Hq, Hkv, Hkv)]
        for dst, src in zip((q, k, v), x):
            dst.copy_(src)
        graph.replay()
        assert granted.tolist() == [1] * B
        sk.kv_append(table, ring, x[0], x[1], x[2])
        want = sk.decode_attention(ring, x[0][:, 0].contiguous())
        # the same rows in another order: weights and sums are rounded in another order, each
        # weight to 11 bits, and the outputs to bf16
        assert (out.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max() + 2.0 ** -9
    assert P.error_bits() == 0
