"""Host-side checks of the 4-bit cache entry points: what is refused, and with which
status, before any launch (the pointers below are aligned stand-ins, never read)."""
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


def _layer(sk, k_dtype, v_dtype, k=A, v=None, kind=0, D=128, Hkv=8):
    return sk.KVLayerStruct(kind, k_dtype, v_dtype, 2, Hkv, D, 4, 60, 64, k, v, None, A, A, A, None)


def _paged(sk, k_dtype, v_dtype, k=A, v=None, D=128):
    return sk.PagedLayerStruct(k_dtype, v_dtype, 2, 8, D, 16, 4, 0, 0, 0, 16, k, v, A, None, A, None)


def test_row_bytes():
    import sink_kv_attention_gb300 as sk
    assert sk.kv4_row_bytes(128) == 160 and sk.kv4_row_bytes(64) == 80


def test_append_refusals(lib):
    import sink_kv_attention_gb300 as sk

    def append(L, io=sk.SK_BF16, T=1, k=A):
        return lib.sk_kv_append(None, ctypes.byref(L), None, 0, k, A, io, T, None)

    I4, BF = sk.SK_I4, sk.SK_BF16
    assert append(_layer(sk, I4, I4), T=0) == sk.SK_OK
    assert append(_layer(sk, I4, I4, v=A), T=0) == sk.SK_ERR_ARG        # V rows are in k
    assert append(_layer(sk, I4, I4, k=None), T=0) == sk.SK_ERR_ARG
    assert append(_layer(sk, I4, BF, v=A), T=0) == sk.SK_ERR_ARG        # both or neither
    assert append(_layer(sk, BF, I4, v=A), T=0) == sk.SK_ERR_ARG
    assert append(_layer(sk, BF, BF), T=0) == sk.SK_ERR_ARG             # bf16 wants a V buffer
    assert append(_layer(sk, I4, I4, k=A + 8), T=0) == sk.SK_ERR_ARG    # alignment
    assert append(_layer(sk, I4, I4), io=sk.SK_I8) == sk.SK_ERR_UNSUPPORTED
    assert append(_layer(sk, I4, I4, D=96)) == sk.SK_ERR_UNSUPPORTED


def test_attention_refusals(lib):
    import sink_kv_attention_gb300 as sk
    I4 = sk.SK_I4

    def attend(L, Hq=32, io=sk.SK_BF16, q=A, ws=1 << 30):
        return lib.sk_decode_attention(ctypes.byref(L), q, Hq, io, None, A, A, ws, None)

    good = _layer(sk, I4, I4)
    assert attend(good, Hq=24) == sk.SK_ERR_UNSUPPORTED                 # 3 q heads per kv head
    assert attend(good, Hq=33) == sk.SK_ERR_ARG
    assert attend(good, Hq=128) == sk.SK_ERR_UNSUPPORTED                # 16 per kv head
    assert attend(good, io=sk.SK_I8) == sk.SK_ERR_UNSUPPORTED
    assert attend(good, q=A + 4) == sk.SK_ERR_ARG
    assert attend(good, ws=64) == sk.SK_ERR_ARG
    assert attend(_layer(sk, I4, I4, D=96)) == sk.SK_ERR_UNSUPPORTED
    assert attend(_layer(sk, I4, I4, v=A)) == sk.SK_ERR_ARG
    for D in (64, 128):
        for rep in (1, 2, 4, 8):
            L = _layer(sk, I4, I4, D=D)
            assert lib.sk_decode_workspace_bytes(ctypes.byref(L), 8 * rep) > 0
            Lp = _paged(sk, I4, I4, D=D)
            assert lib.sk_paged_decode_workspace_bytes(ctypes.byref(Lp), 8 * rep) > 0
    assert lib.sk_decode_workspace_bytes(ctypes.byref(good), 24) == 0
    bad = _paged(sk, I4, I4, v=A)
    assert lib.sk_paged_decode_workspace_bytes(ctypes.byref(bad), 32) == 0
    assert lib.sk_paged_decode_attention(ctypes.byref(bad), A, 32, sk.SK_BF16, None, A, A, 1 << 30, None) == \
        sk.SK_ERR_ARG
    mixed = _paged(sk, I4, sk.SK_BF16, v=A)
    assert lib.sk_paged_decode_workspace_bytes(ctypes.byref(mixed), 32) == 0


def test_workspace_holds_either_way_of_pairing_kv_heads(lib):
    """A slot (a mark of 8 bytes and HEADS (D + 2) floats, padded to 16 bytes) for each unit and
    block, whether a unit has one kv head (fp32 calls) or two; without a device the block
    count is 1."""
    import sink_kv_attention_gb300 as sk
    for D in (64, 128):
        for rep in (1, 2, 4, 8):
            for Hkv in (1, 2, 32):
                L = _layer(sk, sk.SK_I4, sk.SK_I4, D=D, Hkv=Hkv)
                L.batch = 1024
                got = lib.sk_decode_workspace_bytes(ctypes.byref(L), Hkv * rep)
                for kvh in (1, 2):
                    if kvh == 2 and (rep > 4 or Hkv % 2):
                        continue
                    slots = 1024 * Hkv // kvh + 1
                    assert got >= slots * 8 + slots * 4 * ((kvh * rep * (D + 2) + 3) // 4 * 4), (D, rep, Hkv, kvh)


def test_sizes_past_32_bit_shares_are_refused(lib):
    import sink_kv_attention_gb300 as sk
    P = _paged(sk, sk.SK_I4, sk.SK_I4)
    P.max_blocks, P.block_size = (1 << 31) - 1, 1024
    assert lib.sk_paged_decode_attention(ctypes.byref(P), A, 32, sk.SK_BF16, None, A, A, 1 << 40, None) == \
        sk.SK_ERR_UNSUPPORTED


def test_other_entry_points_refuse_4_bit_layers(lib):
    """The fused decode step, rerotation and shift have no 4-bit form."""
    import sink_kv_attention_gb300 as sk
    L = _layer(sk, sk.SK_I4, sk.SK_I4)
    assert lib.sk_decode_step_workspace_bytes(ctypes.byref(L), 32) == 0
    assert lib.sk_decode_step(None, ctypes.byref(L), A, 32, A, A, sk.SK_BF16, None, A, A, 1 << 30, None) == \
        sk.SK_ERR_UNSUPPORTED


def test_unpack_refusals(lib):
    import sink_kv_attention_gb300 as sk
    f = lib.sk_kv4_unpack
    assert f(None, 0, 128, None, None, sk.SK_BF16, None) == sk.SK_OK
    assert f(A, -1, 128, A, A, sk.SK_BF16, None) == sk.SK_ERR_ARG
    assert f(None, 1, 128, A, A, sk.SK_BF16, None) == sk.SK_ERR_ARG
    assert f(A, 1, 128, A + 8, A, sk.SK_BF16, None) == sk.SK_ERR_ARG
    assert f(A, 1, 96, A, A, sk.SK_BF16, None) == sk.SK_ERR_UNSUPPORTED
    assert f(A, 1, 128, A, A, sk.SK_I8, None) == sk.SK_ERR_UNSUPPORTED
    assert f(A, 1, 128, A, A, sk.SK_I4, None) == sk.SK_ERR_UNSUPPORTED


def test_python_checks():
    import sink_kv_attention_gb300 as sk
    with pytest.raises(ValueError):
        sk.KVLayer.allocate(sk.SK_LAYER_RING, 1, 1, 64, sinks=1, window=3, device="cpu", bits=8)
    with pytest.raises(ValueError):
        sk.PagedLayer.allocate(1, 1, 64, block_size=16, n_blocks=2, max_blocks=2, device="cpu", bits=2)
    with pytest.raises(TypeError):
        sk.kv4_unpack(torch.zeros(3, 80))
    with pytest.raises(ValueError):
        sk.kv4_unpack(torch.zeros(3, 82, dtype=torch.uint8))
    with pytest.raises(ValueError):
        sk.kv4_unpack(torch.zeros(3, 160, dtype=torch.uint8)[:, ::2])
    with pytest.raises(ValueError):      # a row that is no 4-bit row
        sk.KVLayer(sk.SK_LAYER_GLOBAL, torch.zeros(1, 1, 4, 161, dtype=torch.uint8), None, torch.zeros(1).long()).struct()
    L = sk.KVLayer.allocate(sk.SK_LAYER_RING, 2, 3, 128, sinks=1, window=3, device="cpu", bits=4)
    assert L.k.shape == (2, 3, 4, 160) and L.k.dtype == torch.uint8 and L.v is None and L.head_dim == 128
    s = L.struct()
    assert (s.k_dtype, s.v_dtype, s.v, s.head_dim) == (sk.SK_I4, sk.SK_I4, None, 128)
    P = sk.PagedLayer.allocate(2, 3, 64, block_size=16, n_blocks=5, max_blocks=2, device="cpu", bits=4)
    s = P.struct()
    assert P.k_pool.shape == (5, 3, 16, 80) and (s.k_dtype, s.v_pool, s.head_dim) == (sk.SK_I4, None, 64)
