"""What the cache operators refuse before anything is launched, on the CPU:
argument checks come before the check of the device, so a host-only layout and
pointers that are never followed reach every one of them."""
import ctypes

import pytest

import block_sparse_long_bsa_b200 as bsa
from oracle import layouts as OL

INVALID, SHAPE, UNSUPPORTED = 1, 2, 3
N, B = 1000, 64
P = 1 << 20          # an aligned address that no refused call follows


@pytest.fixture(scope="module")
def lay():
    from block_sparse_long_bsa_b200 import build
    build.build()
    lay = bsa.Layout(OL.DYADIC, N, B, 2, -1, window=2, global_first=1, dyadic_kmin=2)
    yield lay
    lay.close()


def _status(call, args):
    with pytest.raises(bsa.BsaError) as e:
        call(*args.values())
    return e.value.status


def _weights_args(lay, **bad):
    args = dict(q=P, k=P, lse=P, layout=lay.handle, B=B, n=N, heads=8, kv_heads=4, d=64, scale=0.1, weights=P,
                stride=N, workspace=P, size=1 << 40)
    args.update(bad)
    return args


def _step_args(lay, **bad):
    args = dict(q=P, kc=P, vc=P, table=P, max_blocks=16, num_pages=32, positions=P, layout=lay.handle, batch=2, heads=8,
                kv_heads=4, d=64, scale=0.1, o=P, lse=P, weights=P, stride=N, workspace=P, size=1 << 40)
    args.update(bad)
    return args


def _evict_args(lay, **bad):
    args = dict(kc=P, vc=P, table=P, max_blocks=16, num_pages=32, lengths=P, weights=P, tokens=P, layout=lay.handle,
                batch=2, kv_heads=4, d=64, budget=100, recent=10, stride=N, weights_out=2 * P, tokens_out=3 * P,
                lengths_out=4 * P, workspace=P, size=1 << 40)
    args.update(bad)
    return args


def _tree_args(lay, **bad):
    args = dict(q=P, kt=P, vt=P, kc=P, vc=P, table=P, max_blocks=16, num_pages=32, lengths=P, parents=P,
                layout=lay.handle, T=8, batch=2, heads=8, kv_heads=4, d=64, scale=0.1, o=P, lse=P, workspace=P,
                size=1 << 40)
    args.update(bad)
    return args


CALLS = {"weights": (bsa.bsa_attention_weights, _weights_args), "step": (bsa.bsa_decode_weights, _step_args),
         "evict": (bsa.bsa_evict, _evict_args), "tree": (bsa.bsa_decode_tree, _tree_args)}

BAD = [
    ("weights", dict(B=128), SHAPE), ("weights", dict(n=N - 1), SHAPE), ("weights", dict(stride=N - 1), SHAPE),
    ("weights", dict(heads=6, kv_heads=4), SHAPE), ("weights", dict(heads=3, kv_heads=1), SHAPE),
    ("weights", dict(q=P + 8), INVALID), ("weights", dict(weights=P + 2), INVALID), ("weights", dict(lse=0), INVALID),
    ("step", dict(stride=N - 1), SHAPE), ("step", dict(max_blocks=15), SHAPE), ("step", dict(num_pages=0), SHAPE),
    ("step", dict(num_pages=(1 << 31) - 1), SHAPE), ("step", dict(positions=0), INVALID),
    ("step", dict(kc=P + 8), INVALID), ("step", dict(weights=0), INVALID), ("step", dict(heads=7), SHAPE),
    ("evict", dict(budget=0), SHAPE), ("evict", dict(recent=-1), SHAPE), ("evict", dict(recent=101), SHAPE),
    ("evict", dict(stride=N - 1), SHAPE), ("evict", dict(max_blocks=15), SHAPE), ("evict", dict(num_pages=0), SHAPE),
    ("evict", dict(weights_out=P), INVALID), ("evict", dict(tokens_out=P), INVALID),
    ("evict", dict(lengths_out=P), INVALID), ("evict", dict(kv_heads=3), SHAPE), ("evict", dict(kc=P + 8), INVALID),
    ("evict", dict(lengths=P + 2), INVALID),
    ("tree", dict(T=0), UNSUPPORTED), ("tree", dict(T=129), UNSUPPORTED), ("tree", dict(parents=0), INVALID),
    ("tree", dict(kt=P + 8), INVALID), ("tree", dict(vt=0), INVALID), ("tree", dict(max_blocks=15), SHAPE),
    ("tree", dict(heads=4, kv_heads=8), SHAPE), ("tree", dict(parents=P + 1), INVALID),
] + [(name, bad, code) for name in CALLS for bad, code in (
    (dict(layout=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(workspace=0), INVALID), (dict(workspace=P + 8), INVALID),
    (dict(size=1), SHAPE))
] + [(name, bad, code) for name in ("weights", "step", "tree") for bad, code in (
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(heads=0), SHAPE), (dict(kv_heads=0), SHAPE))
] + [(name, dict(batch=0), SHAPE) for name in ("step", "evict", "tree")]


@pytest.mark.parametrize("name,bad,code", BAD)
def test_refused(lay, name, bad, code):
    call, args = CALLS[name]
    assert _status(call, args(lay, **bad)) == code


@pytest.mark.parametrize("name", CALLS)
def test_only_the_host_only_layout_is_wrong_with_the_arguments_above(lay, name):
    """Each list of arguments passes every check but the last: so each change above is what was refused."""
    call, args = CALLS[name]
    with pytest.raises(bsa.BsaError, match="host-only"):
        call(*args(lay).values())


def test_an_unsupported_block_size_is_refused():
    odd = bsa.Layout(OL.BAND_GLOBAL, 100, 32, 1, -1, window=1, global_first=0)
    for name, (call, args) in CALLS.items():
        bad = dict(B=32, n=100) if name == "weights" else {}
        assert _status(call, args(odd, **bad)) == UNSUPPORTED
    odd.close()


def test_workspace_sizes(lay):
    """0 where the call is refused, else what the stated parts take."""
    h = lay.handle
    assert bsa.bsa_attention_weights_workspace_bytes(0, 8, 4) == 0
    assert bsa.bsa_attention_weights_workspace_bytes(h, 6, 4) == 0
    row_ptr, _ = bsa.bsa_layout_csr(h)
    nb = len(row_ptr) // 2
    kept = max(row_ptr[nb] - row_ptr[0], row_ptr[2 * nb] - row_ptr[nb])
    assert bsa.bsa_attention_weights_workspace_bytes(h, 8, 4) == 8 * kept * B * 4
    assert bsa.bsa_evict_workspace_bytes(h, 2, 4, 0) == 0
    assert bsa.bsa_evict_workspace_bytes(h, 2, 4, 100) >= 4 * 100 * 4 * 2
    # a budget past the layout's tokens needs no more than one of all of them
    assert bsa.bsa_evict_workspace_bytes(h, 2, 4, 1 << 30) == bsa.bsa_evict_workspace_bytes(h, 2, 4, N)
    assert bsa.bsa_decode_weights_workspace_bytes(h, 2, 8, 4, 96) == 0
    assert bsa.bsa_decode_weights_workspace_bytes(h, 2, 8, 4, 64) > 0
    assert bsa.bsa_decode_tree_workspace_bytes(h, 2, 8, 4, 129, 64) == 0
    small, large = (bsa.bsa_decode_tree_workspace_bytes(h, 2, 8, 4, T, 64) for T in (1, 128))
    assert 0 < small < large


def test_prompt_weights_take_as_many_heads_at_a_time_as_64_mib_hold():
    n = 64 * 600
    for heads, kv, units in ((8, 4, 1), (9, 3, 3), (2, 2, 1)):
        full = bsa.Layout(OL.BAND_GLOBAL, n, 64, 1, -1, window=600, global_first=0)
        one = units * (600 * 601 // 2) * 64 * 4
        need = bsa.bsa_attention_weights_workspace_bytes(full.handle, heads, kv)
        assert need == max(1, min(kv, (64 << 20) // one)) * one
        full.close()


def test_sizes_that_pass_32_bits_are_refused_not_wrapped(lay):
    assert bsa.bsa_decode_tree_workspace_bytes(lay.handle, 1, 1 << 30, 2, 128, 64) == 0
    assert bsa.bsa_evict_workspace_bytes(lay.handle, 1, (1 << 31) - 1, 10) == 0
    assert bsa.bsa_attention_weights_workspace_bytes(lay.handle, (1 << 30), 1 << 30) == 0
    assert ctypes.sizeof(ctypes.c_size_t) == 8


def test_the_conveniences_refuse_a_host_only_layout_as_the_calls_do():
    torch = pytest.importorskip("torch")
    only = bsa.Layout(OL.BAND_GLOBAL, 200, 64, 1, -1, window=4, global_first=0)
    q, k, lse = torch.zeros((2, 200, 64)).bfloat16(), torch.zeros((1, 200, 64)).bfloat16(), torch.zeros((2, 200))
    cache, table, one = torch.zeros((4, 1, 64, 64)).bfloat16(), torch.zeros((1, 4)).int(), torch.zeros(1).int()
    w, row, tree = torch.zeros((1, 200)), q[:, 0].contiguous(), q[:, :3].contiguous()
    own = torch.zeros(1 << 16, dtype=torch.uint8)
    for more in ({}, {"workspace": own}):
        for call in (lambda: bsa.attention_weights(q, k, lse, only, **more),
                     lambda: bsa.decode_weights(row, cache, cache, table, one, only, 1, w, **more),
                     lambda: bsa.evict(cache, cache, table, one, w, only, 100, **more),
                     lambda: bsa.decode_tree(tree, k[:, :3].contiguous(), k[:, :3].contiguous(), cache, cache, table, one,
                                             torch.zeros((1, 3)).int() - 1, only, **more)):
            with pytest.raises(bsa.BsaError, match="host-only") as e:
                call()
            assert e.value.status == INVALID
    only.close()


def test_the_cut_refuses_layouts_past_2_to_the_30():
    """Its threads step through the slots with 32-bit numbers; the caches of so many tokens would pass the GPU's memory."""
    n = (1 << 30) + 1
    long = bsa.Layout(OL.BAND_GLOBAL, n, 128, 1, -1, window=0, global_first=0)
    assert bsa.bsa_evict_workspace_bytes(long.handle, 1, 1, 10) == 0
    assert _status(bsa.bsa_evict, _evict_args(long, max_blocks=1 << 24, stride=n, batch=1, kv_heads=1)) == SHAPE
    long.close()
