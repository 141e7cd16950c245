"""The calls of several sequences refuse what they do not document, on the host
and before any launch (no GPU needed)."""

import pytest

INVALID, CAPACITY = 1, 3
P = 0x10000  # 256-byte aligned addresses that are never read here
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from self_speculative_decoding_gb300 import build as b
    b.build()
    from self_speculative_decoding_gb300 import _abi
    return _abi.load()


ONE = 2 * 256 * 64                    # Hkv rows dh
ROPE = dict(qkv=MB, B=2, T=4, lengths=P, counts=P, positions=P, q_gain=P, k_gain=P, eps=1e-5, theta=1e4,
            k=16 * MB, v=32 * MB, rows=256, stride=ONE, H=4, Hkv=2, dh=64, q_out=2 * MB, stream=None)


@pytest.mark.parametrize("change", [
    dict(qkv=None), dict(qkv=MB + 8), dict(B=0), dict(B=513), dict(T=0), dict(T=257), dict(H=65536, T=256, B=512, dh=128, rows=2**20, stride=2**40), dict(lengths=None),
    dict(lengths=P + 2), dict(counts=P + 1), dict(positions=P + 1), dict(q_gain=P + 4), dict(k_gain=P + 8),
    dict(eps=-1.0), dict(eps=float("nan")), dict(theta=0.0), dict(theta=float("inf")), dict(k=None),
    dict(v=32 * MB + 8), dict(rows=0), dict(stride=ONE - 8), dict(stride=ONE + 4), dict(H=0), dict(Hkv=0),
    dict(dh=96), dict(q_out=None), dict(q_out=MB + 256), dict(v=16 * MB), dict(v=16 * MB + 4096),
    dict(qkv=16 * MB), dict(q_out=32 * MB), dict(lengths=2 * MB), dict(positions=16 * MB + 4), dict(k_gain=32 * MB)])
def test_rope_append(lib, change):
    assert lib.ssd_op_rope_append(*{**ROPE, **change}.values()) == INVALID
    assert b"rope_append" in lib.ssd_ops_last_error()


QUANT = dict(k=16 * MB, v=32 * MB, rows=256, stride=ONE, held=P, lengths=P, B=2, Hkv=2, dh=64, block=64,
             k8=48 * MB, v8=64 * MB, ks=80 * MB, vs=96 * MB, max_seq=512, stride8=2 * ONE, sstride=16,
             held_out=P + 4096, stream=None)


@pytest.mark.parametrize("change", [
    dict(k=None), dict(v=32 * MB + 8), dict(rows=0), dict(stride=ONE - 8), dict(held=None), dict(lengths=None),
    dict(B=0), dict(Hkv=0), dict(dh=32), dict(block=16), dict(block=48), dict(block=256), dict(max_seq=500),
    dict(max_seq=0), dict(k8=None), dict(v8=64 * MB + 8), dict(ks=None), dict(vs=96 * MB + 2),
    dict(stride8=2 * ONE - 16), dict(stride8=2 * ONE + 8), dict(sstride=15), dict(held_out=None),
    dict(held_out=P), dict(held_out=P + 4), dict(v8=48 * MB + 65536), dict(vs=80 * MB + 32),
    dict(k8=16 * MB), dict(v8=32 * MB + 4096), dict(ks=16 * MB), dict(vs=64 * MB),
    dict(held=80 * MB), dict(held_out=48 * MB), dict(held_out=96 * MB)])
def test_cache_quantize(lib, change):
    assert lib.ssd_op_cache_quantize(*{**QUANT, **change}.values()) == INVALID
    assert b"cache_quantize" in lib.ssd_ops_last_error()


ATTN = dict(q=MB, B=2, T=4, lengths=P, counts=P, k=16 * MB, v=32 * MB, rows=256, stride=ONE, k8=48 * MB,
            v8=64 * MB, ks=80 * MB, vs=96 * MB, held=P, max_seq=512, block=64, stride8=2 * ONE, sstride=16,
            window=0, sinks=0, H=4, Hkv=2, dh=64, scale=0.125, out=2 * MB, ws=128 * MB, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=MB + 8), dict(B=0), dict(B=513), dict(T=0), dict(T=65), dict(H=3), dict(H=0),
    dict(H=258), dict(Hkv=0), dict(dh=96), dict(lengths=None), dict(counts=P + 1), dict(k=None),
    dict(v=None), dict(rows=0), dict(stride=ONE - 8), dict(k8=None), dict(v8=None), dict(ks=None),
    dict(vs=None), dict(held=None), dict(held=P + 2), dict(max_seq=500), dict(block=96), dict(stride8=16),
    dict(sstride=1), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(out=None),
    dict(out=2 * MB + 8), dict(ws=None), dict(ws=128 * MB + 16),
    dict(out=MB), dict(out=16 * MB), dict(out=64 * MB), dict(out=96 * MB), dict(out=128 * MB + 256), dict(lengths=2 * MB + 4),
    dict(ws=MB), dict(ws=32 * MB), dict(ws=48 * MB), dict(ws=80 * MB), dict(ws=P)])
def test_cache_attention(lib, change):
    assert lib.ssd_op_cache_attention(*{**ATTN, **change}.values()) == INVALID
    assert b"cache_attention" in lib.ssd_ops_last_error()


def test_small_workspaces(lib):
    need = lib.ssd_op_cache_attention_workspace(2, 4, 4, 2, 64)
    assert need > 0
    assert lib.ssd_op_cache_attention(*{**ATTN, "ws_bytes": need - 1}.values()) == CAPACITY
    for bad in ((0, 4, 4, 2, 64), (2, 65, 4, 2, 64), (2, 4, 4, 3, 64), (2, 4, 4, 2, 80)):
        assert lib.ssd_op_cache_attention_workspace(*bad) == 0


def test_cache_give_up(lib):
    assert lib.ssd_debug_cache_give_up(-2) == INVALID
    assert b"cache_give_up" in lib.ssd_ops_last_error()
    assert lib.ssd_debug_cache_give_up(3) == 0 and lib.ssd_debug_cache_give_up(-1) == 0


VERIFY = dict(p=MB, q=2 * MB, drafts=P, counts=P, au=P, su=P, B=2, d=4, V=100, tokens=P + 4096, n=P + 8192,
              stream=None)


@pytest.mark.parametrize("change", [
    dict(p=None), dict(p=MB + 2), dict(q=2 * MB + 1), dict(drafts=None), dict(counts=P + 1), dict(au=None),
    dict(su=None), dict(B=0), dict(B=513), dict(d=-1), dict(d=1025), dict(V=0), dict(V=2**30 + 1), dict(tokens=None),
    dict(n=None), dict(n=P + 1), dict(tokens=P), dict(tokens=P + 28), dict(tokens=P + 8192),
    dict(tokens=MB), dict(n=2 * MB), dict(n=P + 4), dict(counts=P + 4100)])
def test_verify_drafts(lib, change):
    assert lib.ssd_op_verify_drafts(*{**VERIFY, **change}.values()) == INVALID
    assert b"verify_drafts" in lib.ssd_ops_last_error()
