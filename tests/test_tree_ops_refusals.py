"""The tree-decoding calls refuse what they do not document, on the host and
before any launch (no GPU needed)."""

import pytest

INVALID, CAPACITY = 1, 3
P = 0x10000  # 256-byte aligned addresses that are never read here


@pytest.fixture(scope="module")
def lib():
    from self_speculative_decoding_gb300 import build as b
    b.build()
    from self_speculative_decoding_gb300 import _abi
    return _abi.load()


TREE = dict(qkv=P, parents=P, T=4, n=10, pos0=10, k=1 << 24, v=1 << 25, max_seq=64, H=4, Hkv=2, dh=64,
            theta=1e4, w_in=None, w_out=None, out=P, ws=P, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change", [
    dict(T=0), dict(T=1025), dict(n=-1), dict(n=61), dict(n=2**31 - 1), dict(pos0=-1),
    dict(pos0=2**31 - 2), dict(max_seq=0), dict(H=0), dict(Hkv=0), dict(H=3), dict(dh=96),
    dict(theta=0.0), dict(theta=float("nan")), dict(theta=float("inf")), dict(qkv=None),
    dict(qkv=P + 4), dict(parents=None), dict(parents=P + 2), dict(k=None), dict(v=(1 << 25) + 8),
    dict(out=None), dict(ws=None), dict(ws=P + 16), dict(w_in=P), dict(w_out=P + 2),
    dict(w_in=P + 1, w_out=P), dict(v=1 << 24), dict(v=(1 << 24) + 8192), dict(k=(1 << 25) - 256),
    dict(w_in=P, w_out=P + 256), dict(w_in=P + 508, w_out=P)])
def test_tree_attention(lib, change):
    a = {**TREE, **change}
    assert lib.ssd_op_tree_attention(*a.values()) == INVALID
    assert b"tree_attention" in lib.ssd_ops_last_error()


def test_small_workspaces(lib):
    need = lib.ssd_op_tree_attention_workspace(4, 10, 4, 2, 64)
    assert need > 0
    assert lib.ssd_op_tree_attention(*{**TREE, "ws_bytes": need - 1}.values()) == CAPACITY
    assert lib.ssd_op_tree_attention_workspace(0, 10, 4, 2, 64) == 0
    assert lib.ssd_op_tree_attention_workspace(4, 10, 4, 3, 64) == 0
    assert lib.ssd_op_beam_select_workspace(4, 1000, 4) == 0      # needs none
    need = lib.ssd_op_beam_select_workspace(40, 100000, 4)
    assert need > 0
    assert lib.ssd_op_beam_select(*{**SELECT, "ws_bytes": need - 1}.values()) == CAPACITY
    assert lib.ssd_op_beam_select_workspace(4, 0, 4) == 0


MB = 1 << 20
EVICT = dict(k=16 * MB, v=32 * MB, w=P, n=50, keep=20, sinks=2, recent=5, max_seq=64, Hkv=2, dh=64,
             dtype=0, k_out=48 * MB, v_out=64 * MB, w_out=80 * MB, max_out=32, kept=P, stream=None)


@pytest.mark.parametrize("change", [
    dict(n=0), dict(n=65), dict(keep=0), dict(keep=51, max_out=64), dict(keep=33), dict(sinks=-1),
    dict(recent=-1), dict(sinks=16), dict(sinks=2**31 - 1), dict(Hkv=0), dict(Hkv=65536),
    dict(dh=4), dict(dh=0), dict(dtype=2), dict(k=None), dict(v=32 * MB + 8), dict(w=None),
    dict(w=P + 2), dict(kept=None), dict(k_out=None), dict(v_out=None), dict(w_out=80 * MB + 1),
    dict(k_out=16 * MB), dict(v_out=48 * MB + 1024), dict(k_out=32 * MB + 4096), dict(w_out=P)])
def test_cache_evict(lib, change):
    assert lib.ssd_op_cache_evict(*{**EVICT, **change}.values()) == INVALID
    assert b"cache_evict" in lib.ssd_ops_last_error()


SELECT = dict(logits=P, B=40, V=100000, lse=P, stride=1, scores=P, done=P, end_id=2, W=4, tokens=P,
              parents=P, scores_out=P, done_out=P, ws=P, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change", [
    dict(B=0), dict(B=257), dict(V=0), dict(W=0), dict(W=257), dict(stride=0), dict(end_id=-2),
    dict(end_id=100000), dict(end_id=-1), dict(logits=None), dict(logits=P + 2), dict(scores=None),
    dict(lse=P + 1), dict(done=P + 1), dict(tokens=None), dict(parents=None),
    dict(scores_out=None), dict(done_out=P + 1), dict(ws=None), dict(ws=P + 8)])
def test_beam_select(lib, change):
    assert lib.ssd_op_beam_select(*{**SELECT, **change}.values()) == INVALID
    assert b"beam_select" in lib.ssd_ops_last_error()


REORDER = dict(k=16 * MB, v=32 * MB, parents=P, B=2, W=2, groups=4, max_seq=64, start=3, stop=9,
               row_bytes=128, k_out=48 * MB, v_out=64 * MB, stream=None)


@pytest.mark.parametrize("change", [
    dict(B=0), dict(W=0), dict(groups=0), dict(max_seq=0), dict(start=-1), dict(start=10),
    dict(stop=65), dict(row_bytes=0), dict(row_bytes=24), dict(k=None), dict(k_out=None),
    dict(v=None), dict(v_out=None), dict(v=32 * MB + 8), dict(parents=None), dict(parents=P + 1),
    dict(k_out=16 * MB + 4096), dict(v_out=32 * MB), dict(v_out=48 * MB), dict(k_out=32 * MB)])
def test_beam_reorder(lib, change):
    assert lib.ssd_op_beam_reorder(*{**REORDER, **change}.values()) == INVALID
    assert b"beam_reorder" in lib.ssd_ops_last_error()


def test_an_empty_range_is_no_call(lib):
    assert lib.ssd_op_beam_reorder(*{**REORDER, "start": 9}.values()) == 0


def test_workspaces_of_the_largest_sizes(lib):
    """n_ctx + T and V up to 2^31 - 1: sizes that are whole, or 0 where the call
    refuses them."""
    tree = lib.ssd_op_tree_attention_workspace
    sizes = [tree(1, n, 4, 2, 64) for n in (10, 2**30, 2**31 - 200, 2**31 - 100, 2**31 - 2)]
    assert sizes == sorted(sizes) and 0 < sizes[0] and sizes[-1] < 2**37
    assert tree(1, 2**31 - 1, 4, 2, 64) == 0
    assert tree(1024, 2**31 - 1024, 4, 2, 64) == 0 and tree(1024, 2**31 - 1025, 4, 2, 64) > 0


@pytest.mark.parametrize("T,n,H,Hkv,dh", [(1024, 0, 64, 8, 128), (5, 83, 40, 40, 64), (300, 100, 32, 32, 128)])
def test_workspace_of_one_split_holds_no_partial_outputs(lib, T, n, H, Hkv, dh):
    q = (2 * T * H + 2 * T * Hkv) * dh * 2               # two planes of q, the tree's K and V rows
    rows, blocks = T * H // Hkv, -(-n // 128) + -(-T // 128)
    scores = Hkv * blocks * rows * 512 if rows <= 32 else 0
    small = T * (4 * -(-T // 128) + 2) * 4 + Hkv * (T + 3) + 4 * T * H
    assert lib.ssd_op_tree_attention_workspace(T, n, H, Hkv, dh) <= q + scores + small + 10 * 256


def test_workspaces_of_the_largest_vocabularies(lib):
    # a list of W keys of 8 bytes for each piece of at most 22528 logits
    for V in (2**30, 2**31 - 22528, 2**31 - 10000, 2**31 - 1):
        assert lib.ssd_op_beam_select_workspace(256, V, 7) == 256 * -(-V // 22528) * 7 * 8


def test_binding_refuses_tensors_it_cannot_take():
    import torch
    from self_speculative_decoding_gb300 import ops
    f, i = torch.zeros(4, 8 * 64), torch.zeros(4, dtype=torch.int32)
    c = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):       # host tensors
        ops.tree_attention(f, i, c, c, 10, 10, 4, 2, 64, 1e4)
    with pytest.raises(ValueError):       # parents of another type
        ops.tree_attention(f, i.long(), c, c, 10, 10, 4, 2, 64, 1e4)
    with pytest.raises(ValueError):       # too few columns
        ops.tree_attention(f[:, :-1], i, c, c, 10, 10, 4, 2, 64, 1e4)
    with pytest.raises(ValueError):
        ops.cache_evict(c.half(), c, torch.zeros(2, 64), 10, 5, c, c)
    with pytest.raises(ValueError):
        ops.cache_evict(c, c, torch.zeros(2, 63), 10, 5, c, c)
    with pytest.raises(ValueError):
        ops.beam_select(f, torch.zeros(3), 4)
    with pytest.raises(ValueError):
        ops.beam_reorder(c, None, i, 0, 4, c, c)


def test_binding_refuses_arguments_of_other_types():
    import torch
    from self_speculative_decoding_gb300 import ops
    f, i = torch.zeros(4, 8 * 64), torch.zeros(4, dtype=torch.int32)
    c = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    for bad in (2 ** 31, -2 ** 31 - 1, 2 ** 70):      # would not reach the kernels whole
        with pytest.raises(ValueError, match="32 bits"):
            ops.tree_attention(f, i, c, c, bad, 10, 4, 2, 64, 1e4)
        with pytest.raises(ValueError, match="32 bits"):
            ops.cache_evict(c, c, torch.zeros(2, 64), bad, 5, c, c)
        with pytest.raises(ValueError, match="32 bits"):
            ops.beam_select(f, torch.zeros(4), bad)
        with pytest.raises(ValueError, match="32 bits"):
            ops.beam_reorder(c, None, i, 0, bad, c, None)
    with pytest.raises(TypeError):
        ops.beam_select(f, torch.zeros(4), 2.5)
    with pytest.raises(TypeError):
        ops.tree_attention(f, i, c, c, 10, 10, 4, 2, 64, "theta")
    with pytest.raises(ValueError, match="expected a tensor"):
        ops.cache_evict(None, c, torch.zeros(2, 64), 10, 5, c, c)
    with pytest.raises(ValueError, match="expected a tensor"):
        ops.beam_select(f.numpy(), torch.zeros(4), 2)
    with pytest.raises(ValueError, match="go together"):
        ops.beam_reorder(c, c, i, 0, 4, c, None)
