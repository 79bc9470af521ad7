"""Host-side refusals of the page operations (aligned stand-in pointers, never read)."""
import ctypes
import os

import pytest
import torch

A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    import sink_kv_attention_gb300 as sk
    if not os.path.exists(sk.LIB_PATH):
        from sink_kv_attention_gb300 import build
        build.build()
    return sk._lib()


def _layer(sk, **change):
    f = dict(k_dtype=0, v_dtype=0, batch=2, n_kv_heads=8, head_dim=128, block_size=16, max_blocks=4, n_sink_blocks=0,
             sinks=0, window=0, n_blocks=16, k_pool=A, v_pool=A, block_table=A, sink_block_ids=None, seq_lens=A,
             err=None)
    f.update(change)
    return sk.PagedLayerStruct(**f)


def _calls(lib, sk, layers, n=None, ref=A, other=A, ws=A, ws_bytes=1 << 20):
    arr = (sk.PagedLayerStruct * len(layers))(*layers)
    n = len(layers) if n is None else n
    return [lib.sk_paged_reserve(arr, n, ref, None, other, ws, ws_bytes, None),
            lib.sk_paged_fork(arr, n, ref, other, None),
            lib.sk_paged_compact(arr, n, ref, other, other, ws, ws_bytes, None)]


def test_layers_must_share_a_table(lib):
    import sink_kv_attention_gb300 as sk
    good = _layer(sk)
    for change in (dict(block_table=A + 64), dict(batch=3), dict(max_blocks=5), dict(n_blocks=17), dict(sinks=1),
                   dict(window=9), dict(block_size=32), dict(n_sink_blocks=1, sink_block_ids=A)):
        assert _calls(lib, sk, [good, _layer(sk, **change)]) == [sk.SK_ERR_ARG] * 3, change
    assert _calls(lib, sk, [_layer(sk, k_pool=None)]) == [sk.SK_ERR_ARG] * 3
    assert _calls(lib, sk, [good], n=0) == [sk.SK_ERR_ARG] * 3
    assert _calls(lib, sk, [good] * 129) == [sk.SK_ERR_ARG] * 3
    assert _calls(lib, sk, [good], ref=None) == [sk.SK_ERR_ARG] * 3
    assert _calls(lib, sk, [good], other=None) == [sk.SK_ERR_ARG] * 3
    assert _calls(lib, sk, [_layer(sk, batch=1025)]) == [sk.SK_ERR_UNSUPPORTED] * 3
    assert _calls(lib, sk, [_layer(sk, n_blocks=1 << 31)]) == [sk.SK_ERR_UNSUPPORTED] * 3
    for f in (lib.sk_paged_reserve, lib.sk_paged_compact):
        arr = (sk.PagedLayerStruct * 1)(good)
        for ws, n in ((None, 1 << 20), (A + 8, 1 << 20), (A, 100)):
            assert f(arr, 1, A, A, A, ws, n, None) == sk.SK_ERR_ARG
    assert lib.sk_paged_pages_workspace_bytes(ctypes.byref(good)) > 0
    assert lib.sk_paged_pages_workspace_bytes(None) == 0
    assert lib.sk_paged_pages_workspace_bytes(ctypes.byref(_layer(sk, batch=1025))) == 0


def test_python_checks(lib):
    import sink_kv_attention_gb300 as sk
    with pytest.raises(ValueError):
        sk.PagedGroup([])
    P = sk.PagedLayer.allocate(2, 2, 64, block_size=16, n_blocks=8, max_blocks=3, n_sink_blocks=1, device="cpu")
    g = sk.PagedGroup([P])
    assert g.ref.tolist() == [1] + [0] * 7
    with pytest.raises(ValueError):
        sk.PagedGroup([P], ref=torch.zeros(8))
    with pytest.raises(ValueError):
        sk.PagedGroup([P], ref=torch.zeros(9, dtype=torch.int32))
    with pytest.raises(ValueError):
        g.fork(torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        g.reserve(torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        g.compact(torch.zeros(16, dtype=torch.int32)[::2])
