"""The cache operators' corners on the GPU.  Tolerances as derived in test_gpu_cache.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_sparse_long_bsa_b200 as bsa
from block_sparse_long_bsa_b200 import inputs
from oracle import cache as OC
from oracle import decode as OD
from oracle import layouts as OL

from gpu_common import bf16_half_ulp, to_device_bf16
from test_gpu_cache import DYADIC, _close_lse, _close_o, _close_w, _e_p, _layout, _np, _paged

pytestmark = pytest.mark.gpu

INT_MAX, INT_MIN = 2 ** 31 - 1, -2 ** 31


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bsa.load_library()


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ indices at the ends of 32 bits

@pytest.mark.parametrize("kind,n,L,pat", [
    (OL.DYADIC, 1024, 1, DYADIC),                                             # short rows: one kernel
    (OL.BAND_GLOBAL, 4500, 1, dict(window=71, global_first=0)),               # long rows: two
    (OL.RANDOM, 9000, 4, dict(density=0.6, seed=3)),                          # and a route for each head
])
def test_step_refuses_positions_at_the_ends_of_32_bits(kind, n, L, pat):
    """The largest and the smallest position, as a server may mark a place of the batch that is not in use."""
    B, batch, H, G, d = 64, 4, 4, 2, 64
    lay = _layout(kind, n, B, L, pat)
    kc, vc, table, _ = _paged(batch, G, n, B, d, 300)
    q = to_device_bf16(inputs.normal_bf16_bits((batch * H, d), 301))
    w0 = torch.rand((batch * G, n), device="cuda")
    ref = w0.clone()
    o_ref, lse_ref = bsa.decode_weights(q, kc, vc, table, _i32(5, n - 1, 700, 700), lay, batch, ref)
    w = w0.clone()
    o, lse = bsa.decode_weights(q, kc, vc, table, _i32(INT_MAX, n - 1, INT_MIN, INT_MAX - 1), lay, batch, w)
    torch.cuda.synchronize()
    with pytest.raises(bsa.BsaError):
        bsa.bsa_get_status(lay.handle)
    for b in range(batch):
        rows, kv = slice(b * H, (b + 1) * H), slice(b * G, (b + 1) * G)
        if b == 1:
            assert torch.equal(o[rows], o_ref[rows]) and torch.equal(lse[rows], lse_ref[rows])
            assert torch.equal(w[kv], ref[kv])
        else:
            assert torch.all(o[rows] == 0) and torch.all(torch.isneginf(lse[rows])) and torch.equal(w[kv], w0[kv])
    lay.close()


@pytest.mark.parametrize("n,budget", [(640, 100), (5000, 2000)])
def test_tree_and_cut_refuse_lengths_at_the_ends_of_32_bits(n, budget):
    B, batch, H, G, d, T = 64, 3, 2, 2, 64, 70
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=n // B + 1, global_first=0))
    kc, vc, table, _ = _paged(batch, G, n, B, d, 310)
    q, kt, vt = (to_device_bf16(x) for x in inputs.qkv_bits(batch * H, batch * G, T, d, seeds=(311, 312, 313)))
    par = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").repeat(batch, 1)
    o_ref, lse_ref = bsa.decode_tree(q, kt, vt, kc, vc, table, _i32(1, 500, 1), par, lay)
    lens = _i32(INT_MAX, 500, INT_MIN)
    o, lse = bsa.decode_tree(q, kt, vt, kc, vc, table, lens, par, lay)
    torch.cuda.synchronize()
    with pytest.raises(bsa.BsaError):
        bsa.bsa_get_status(lay.handle)
    assert torch.equal(o[H:2 * H], o_ref[H:2 * H]) and torch.equal(lse[H:2 * H], lse_ref[H:2 * H])
    for b in (0, 2):
        rows = slice(b * H, (b + 1) * H)
        assert torch.all(o[rows] == 0) and torch.all(torch.isneginf(lse[rows]))
    # parents at the ends refuse their rows and what descends from them
    far = par.clone()
    far[1, 3], far[1, 60] = INT_MAX, INT_MIN
    o, lse = bsa.decode_tree(q, kt, vt, kc, vc, table, _i32(1, 500, 1), far, lay)
    torch.cuda.synchronize()
    with pytest.raises(bsa.BsaError):
        bsa.bsa_get_status(lay.handle)
    assert torch.equal(o[H:2 * H, :3], o_ref[H:2 * H, :3]) and torch.all(torch.isneginf(lse[H:2 * H, 3:]))
    assert torch.equal(o[2 * H:], o_ref[2 * H:])
    w = torch.rand((batch * G, n), device="cuda")
    keys = kc.clone()
    wo, to = torch.full_like(w, 7.0), torch.full(w.shape, 7, dtype=torch.int32, device="cuda")
    _, _, lo = bsa.evict(kc, vc, table, lens, w, lay, budget, 10, weights_out=wo, tokens_out=to)
    torch.cuda.synchronize()
    with pytest.raises(bsa.BsaError):
        bsa.bsa_get_status(lay.handle)
    assert lo.tolist() == [-1, min(500, budget), -1]
    for b in (0, 2):
        rows, mine = slice(b * G, (b + 1) * G), table[b].long()
        assert torch.all(wo[rows] == 7) and torch.all(to[rows] == 7)
        assert torch.equal(kc[mine].view(torch.int16), keys[mine].view(torch.int16))
    lay.close()


# ------------------------------------------------------------------ prompts whose work items are one tile

@pytest.mark.parametrize("B,H,G,d,n,window", [
    (128, 16, 16, 64, 16384, 0),        # one key block a row
    (128, 16, 8, 128, 16384, 0),
    (64, 16, 16, 64, 16000, 1),         # two, a tile
    (64, 32, 16, 128, 16000, 1),        # and two query heads an item
])
def test_prompt_weights_of_rows_of_one_tile(B, H, G, d, n, window):
    """14 and more items a block of threads, each one tile, and an lse of its own for every row, so that an item
    read in another's place shows: every key against fp64, and the same bits every time."""
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=window, global_first=0))
    sets = OL.kept_sets(OL.BAND_GLOBAL, n, B, 1, window=window, global_first=0)
    qb, kb, vb = inputs.qkv_bits(H, G, n, d, seeds=(320, 321, 322))
    q, k, v = (to_device_bf16(x) for x in (qb, kb, vb))
    _, lse = bsa.attention(q, k, v, lay)
    lse += torch.from_numpy(np.random.default_rng(323).uniform(-3, 3, (H, n)).astype(np.float32)).cuda()
    got = [bsa.attention_weights(q, k, lse, lay) for _ in range(6)]
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    assert all(torch.equal(x, got[0]) for x in got)
    qh, kh, lse_h = _np(q), _np(k), _np(lse)
    want = OC.prompt_weights(qh, kh, lse_h, sets, B, d ** -0.5)
    # a thread's longest chain of additions: 2 x 32 of the diagonal, 2 x 8 of the rest, then under 16 joins
    _close_w(_np(got[0]), want, _e_p(d ** -0.5, d, qh, kh, lse_h), lse_h, terms=96)
    lay.close()


def test_prompt_weights_do_not_depend_on_another_calls_time_out():
    """A wait that ran out in another call on the layout stays in its status word until that is read: prompt
    weights are added all the same."""
    n, B, H, G, d = 700, 64, 4, 2, 64
    lay = _layout(OL.DYADIC, n, B, 1, DYADIC)
    q, k, v = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, n, d, seeds=(330, 331, 332)))
    _, lse = bsa.attention(q, k, v, lay)
    want = bsa.attention_weights(q, k, lse, lay)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    bsa.bsa_debug_timeout_probe(lay.handle, d, 2_000_000)
    got = bsa.attention_weights(q, k, lse, lay)
    with pytest.raises(bsa.BsaError) as e:
        bsa.bsa_get_status(lay.handle)
    assert e.value.status == 7 and float(want.min()) > 0 and torch.equal(got, want)
    lay.close()


# ------------------------------------------------------------------ values that meet a probability of zero

# op, tokens of the layout, B, query heads a key/value head (or drafted tokens), d
ZERO = [("step", 1000, 64, 2, 64), ("step", 5000, 64, 2, 128), ("step", 5000, 128, 8, 64), ("step", 3000, 64, 16, 128),
        ("tree", 1000, 64, 3, 64), ("tree", 3000, 128, 5, 128), ("tree", 1000, 64, 40, 128), ("tree", 3000, 128, 70, 64)]


def _zero_case(case, seed):
    op, n, B, m, d = case
    G, H, T = 2, (2 * m if op == "step" else 2), (1 if op == "step" else m)
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=n // B + 1, global_first=0))
    sets = OL.kept_sets(OL.BAND_GLOBAL, n, B, 1, window=n // B + 1, global_first=0)
    kc, vc, table, th = _paged(1, G, n, B, d, seed)
    q, kt, vt = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, T, d, seeds=(seed + 1, seed + 2, seed + 3)))
    end = n - T
    par = np.arange(-1, T - 1, dtype=np.int32)[None]

    def run():
        if op == "step":
            w = torch.zeros((G, n), device="cuda")
            out = bsa.decode_weights(q[:, 0].contiguous(), kc, vc, table, _i32(end - 1), lay, 1, w)
        else:
            out = bsa.decode_tree(q, kt, vt, kc, vc, table, _i32(end), torch.from_numpy(par).cuda(), lay)
        torch.cuda.synchronize()
        bsa.bsa_get_status(lay.handle)
        return [_np(x) for x in out]

    def oracle(values, drafted):
        kh = np.nan_to_num(_np(kc), neginf=-np.inf)
        if op == "step":
            return OD.decode_step(_np(q)[:, 0], kh, values, th, [end - 1], sets, B, d ** -0.5)
        return OC.tree(_np(q), _np(kt), drafted, kh, values, th, [end], par, sets, B, d ** -0.5)

    return lay, q, kt, vt, kc, vc, table, end, run, oracle


@pytest.mark.parametrize("case", ZERO)
def test_large_values_of_keys_without_weight_add_nothing(case):
    """Keys at minus infinity whose values are as large as bf16 holds: all of the first three chunks, a few later
    ones, and a whole chunk in between."""
    op, n, B, m, d = case
    lay, q, kt, vt, kc, vc, table, end, run, oracle = _zero_case(case, 340)
    q[:, :, 1] = q[:, :, 1].abs() + 0.5
    token = torch.arange(-(-n // B) * B, device="cuda")
    out = (token < 192) | (token % 97 == 5) | ((token >= 640) & (token < 704))
    out = out.view(-1, B)[:, None, :]
    pages = table[0].long()
    kc[pages, :, :, 1] = torch.where(out, float("-inf"), kc[pages, :, :, 1])
    vc[pages] = torch.where((out & (token.view(-1, B)[:, None] < end))[..., None], 2.0 ** 127, vc[pages])
    vc[pages, :, :, 0] *= torch.where(out, -1.0, 1.0).to(torch.bfloat16)
    o, lse = run()
    vh, vth = np.nan_to_num(_np(vc)), _np(vt)
    o_ref, lse_ref = oracle(vh, vth)
    o_abs, _ = oracle(np.abs(vh), np.abs(vth))
    assert np.abs(o_ref).max() < 10
    kh = np.nan_to_num(_np(kc), neginf=0).reshape(-1, d)
    e_p = _e_p(d ** -0.5, d, _np(q), np.concatenate([kh, _np(kt).reshape(-1, d)]), lse_ref)
    _close_lse(lse, lse_ref, e_p)
    bound = bf16_half_ulp(o) + 2 * (e_p + 2.0 ** -15) * o_abs
    assert np.all(np.abs(o - o_ref) <= bound), (np.abs(o - o_ref) / bound).max()
    lay.close()


@pytest.mark.parametrize("case", ZERO)
def test_infinite_values_of_equal_keys(case):
    """All probabilities exactly a power of two, so that their second parts are the smallest there are: an infinite
    value still gives an infinity of its sign, and nothing to the other columns."""
    lay, q, kt, vt, kc, vc, table, end, run, oracle = _zero_case(case, 350)
    q.zero_()
    o, _ = run()
    vc[table[0, 1].long(), :, 7, 3], vc[table[0, 2].long(), :, 9, 4] = float("inf"), float("-inf")
    o2, lse2 = run()
    assert np.isfinite(o).all() and np.isfinite(lse2).all()
    assert np.all(o2[..., 3] == np.inf) and np.all(o2[..., 4] == -np.inf)
    o2[..., 3:5] = o[..., 3:5]
    assert np.array_equal(o, o2)
    lay.close()


# ------------------------------------------------------------------ a layout as long as 32 bits count

def test_step_and_tree_at_the_end_of_the_longest_layout():
    """2^31 - 1 tokens, each block for itself: a step at the last position, and a chain whose first token takes it;
    the others lie past the end and are refused."""
    n, B, H, G, d, T = INT_MAX, 128, 2, 1, 64, 5
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=0, global_first=0))
    kc, vc, _, _ = _paged(1, G, B, B, d, 360)
    q, kt, vt = (to_device_bf16(x) for x in inputs.qkv_bits(2 * H, 2 * G, T, d, seeds=(361, 362, 363)))
    table = torch.zeros((2, -(-n // B)), dtype=torch.int32, device="cuda")
    par = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").repeat(2, 1)
    o, lse = bsa.decode_tree(q, kt, vt, kc, vc, table, _i32(n - 1, n), par, lay)
    torch.cuda.synchronize()
    with pytest.raises(bsa.BsaError):
        bsa.bsa_get_status(lay.handle)
    assert torch.all(o[:H, 1:] == 0) and torch.all(torch.isneginf(lse[:H, 1:]))
    assert torch.all(o[H:] == 0) and torch.all(torch.isneginf(lse[H:]))
    end = (n - 1) % B                                # cached tokens of the last block
    page = np.zeros((1, 1), np.int64)
    sets, kh, vh = [[{0}]], _np(kc), _np(vc)
    o_ref, lse_ref = OC.tree(_np(q)[:H, :1], _np(kt)[:G, :1], _np(vt)[:G, :1], kh, vh, page, [end],
                             np.full((1, 1), -1), sets, B, d ** -0.5)
    e_p = _e_p(d ** -0.5, d, _np(q), np.concatenate([kh.reshape(-1, d), _np(kt).reshape(-1, d)]), lse_ref)
    _close_lse(_np(lse)[:H, :1], lse_ref, e_p)
    _close_o(_np(o)[:H, :1], o_ref, e_p, np.concatenate([vh.reshape(-1, d), _np(vt).reshape(-1, d)]))
    w = torch.zeros((G, n), device="cuda")
    row = q[:H, 0].contiguous()
    o, lse = bsa.decode_weights(row, kc, vc, table[:1], _i32(n - 1), lay, 1, w)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    o_ref, lse_ref = OD.decode_step(_np(row), kh, vh, page, [end], sets, B, d ** -0.5)
    e_p = _e_p(d ** -0.5, d, _np(row), kh, lse_ref)
    _close_lse(_np(lse), lse_ref, e_p)
    _close_o(_np(o), o_ref, e_p, vh)
    want = OC.step_weights(_np(row), kh, page, [end], lse_ref, sets, B, d ** -0.5, end + 1)
    bound = want * (2 * e_p + 2.0 ** -21 + H * 2.0 ** -24)
    assert np.all(np.abs(_np(w[:, n - end - 1:]) - want) <= bound)
    assert not torch.any(w[:, :n - end - 1])
    lay.close()


# ------------------------------------------------------------------ running weights read early

@pytest.mark.parametrize("kind,n,B,L,H,G,d,pat", [
    (OL.BAND_GLOBAL, 20000, 64, 1, 4, 2, 64, dict(window=313, global_first=0)),    # two kernels, short rows of queries
    (OL.BAND_GLOBAL, 9000, 128, 1, 32, 2, 64, dict(window=71, global_first=0)),    # 16 query heads a key/value head
    (OL.RANDOM, 9000, 64, 4, 4, 2, 128, dict(density=0.6, seed=3)),                # a route for each head
    (OL.DYADIC, 3000, 64, 1, 4, 2, 128, DYADIC),                                   # one kernel
])
def test_calls_that_follow_each_other_unsynchronised(kind, n, B, L, H, G, d, pat):
    """Steps, trees, prompt weights and torch's own kernels that change the same running weights one after the other, with
    nothing waited for in between: the bits of the same calls with the GPU waited for after each.  Rows of weights
    lie an odd number of floats apart, so that blocks of threads share pieces of memory."""
    batch, prompt = 2, 700
    lay = _layout(kind, n, B, L, pat)
    short = _layout(OL.DYADIC, prompt, B, 1, DYADIC)
    kc, vc, table, _ = _paged(batch, G, n, B, d, 370)
    qp, kp, vp = (to_device_bf16(x) for x in inputs.qkv_bits(batch * H, batch * G, prompt, d, seeds=(371, 372, 373)))
    _, lse_p = bsa.attention(qp, kp, vp, short)
    qs = [to_device_bf16(inputs.normal_bf16_bits((batch * H, d), 380 + i)) for i in range(12)]
    at = [_i32(n - 1 - i, n // 2 + i) for i in range(12)]
    w0 = torch.rand((batch * G, n + 5), device="cuda")
    h = lay.handle
    T = 7
    trees = [[to_device_bf16(x) for x in inputs.qkv_bits(batch * H, batch * G, T, d, seeds=(390 + i, 410 + i, 430 + i))]
             for i in range(12)]
    parents = [_i32(*([-1] + [max(-1, j - 1 - (i + j) % 3) for j in range(1, T)]) * batch).view(batch, T) for i in range(12)]
    ws = torch.empty(max(bsa.bsa_decode_weights_workspace_bytes(h, batch, batch * H, batch * G, d),
                         bsa.bsa_decode_tree_workspace_bytes(h, batch, batch * H, batch * G, T, d),
                         bsa.bsa_attention_weights_workspace_bytes(short.handle, batch * H, batch * G)),
                     dtype=torch.uint8, device="cuda")

    def run(wait):
        w, q, pos, out = w0.clone(), torch.empty_like(qs[0]), torch.empty_like(at[0]), []
        tree = [torch.empty_like(x) for x in trees[0] + [parents[0]]]
        wait()
        for i, (x, t) in enumerate(zip(qs, at)):
            q.copy_(x)
            pos.copy_(t)
            wait()
            for _ in range(2):
                out += bsa.decode_weights(q, kc, vc, table, pos, lay, batch, w, workspace=ws)
                wait()
            for a, b in zip(tree, trees[i] + [parents[i]]):
                a.copy_(b)
            wait()
            out += bsa.decode_tree(*tree[:3], kc, vc, table, pos - T, tree[3], lay, workspace=ws)
            wait()
            if i % 3 == 1:
                w.mul_(0.75)
                wait()
            if i % 4 == 2:
                bsa.attention_weights(qp, kp, lse_p, short, w, workspace=ws)
                wait()
                bsa.attention_weights(qp, kp, lse_p, short, w, workspace=ws)
                wait()
        torch.cuda.synchronize()
        return [w] + out

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        got = run(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    tail = w0[:, n:]
    for _ in range(4):
        tail = tail * 0.75
    assert torch.equal(want[0][:, n:], tail)
    bsa.bsa_get_status(lay.handle)
    bsa.bsa_get_status(short.handle)
    lay.close()
    short.close()


# ------------------------------------------------------------------ shapes between the others

@pytest.mark.parametrize("B,L,H,G,d", [(64, 1, 24, 1, 64), (128, 1, 20, 2, 128), (64, 16, 16, 1, 64), (128, 10, 10, 1, 64)])
def test_prompt_weights_of_many_query_heads_a_key_value_head(B, L, H, G, d):
    """More units a key/value head (12, 10, 16 and 10) than the sum over rows looks up at a time."""
    n, pat = 900, dict(density=0.4, seed=8)
    lay = _layout(OL.RANDOM, n, B, L, pat)
    sets = OL.kept_sets(OL.RANDOM, n, B, L, **pat)
    q, k, v = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, n, d, seeds=(440, 441, 442)))
    _, lse = bsa.attention(q, k, v, lay)
    got = bsa.attention_weights(q, k, lse, lay)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    qh, kh, lse_h = _np(q), _np(k), _np(lse)
    want = OC.prompt_weights(qh, kh, lse_h, sets, B, d ** -0.5)
    # 96 additions in a thread of the first kernel at most, then at most 15 rows of H units
    _close_w(_np(got), want, _e_p(d ** -0.5, d, qh, kh, lse_h), lse_h, terms=96 + 15 * H)
    lay.close()


@pytest.mark.parametrize("n", [1, 2, 40, 63, 64, 65, 128, 190])
@pytest.mark.parametrize("B,H,G,d", [(64, 2, 1, 64), (128, 4, 2, 128), (64, 12, 1, 64)])
def test_steps_over_a_few_tokens(n, B, H, G, d):
    """Rows of one to four chunks, in clusters of one to four, with a page table that is wider than the layout and
    weights that begin at an odd place."""
    batch, wide = 3, -(-n // B) + 3
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=2, global_first=1))
    sets = OL.kept_sets(OL.BAND_GLOBAL, n, B, 1, window=2, global_first=1)
    kc, vc, table, th = _paged(batch, G, n, B, d, 450, spare=2)
    full = torch.full((batch, wide), -9, dtype=torch.int32, device="cuda")
    full[:, :table.shape[1]] = table
    at = [n - 1, n // 2, 0]
    q = to_device_bf16(inputs.normal_bf16_bits((batch * H, d), 451))
    w0 = torch.rand((batch * G, n + 9), device="cuda")
    w = w0.clone()
    o, lse = bsa.decode_weights(q, kc, vc, full, _i32(*at), lay, batch, w[:, 3:3 + n])
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    qh, kh, vh = _np(q), np.nan_to_num(_np(kc)), np.nan_to_num(_np(vc))
    o_ref, lse_ref = OD.decode_step(qh, kh, vh, th, at, sets, B, d ** -0.5)
    e_p = _e_p(d ** -0.5, d, qh, kh, lse_ref)
    _close_lse(_np(lse), lse_ref, e_p)
    _close_o(_np(o), o_ref, e_p, vh)
    want = OC.step_weights(qh, kh, th, at, lse_ref, sets, B, d ** -0.5, n)
    base = _np(w0[:, 3:3 + n])
    bound = want * (2 * e_p + 2.0 ** -21 + H // G * 2.0 ** -24) + 2.0 ** -24 * (want + base)
    assert np.all(np.abs(_np(w[:, 3:3 + n]) - base - want) <= bound)
    w[:, 3:3 + n] = w0[:, 3:3 + n]
    assert torch.equal(w, w0)
    lay.close()


@pytest.mark.parametrize("op,n,m", [("step", 1000, 2), ("step", 5000, 2), ("step", 3000, 16), ("tree", 1000, 3), ("tree", 3000, 40)])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_a_query_that_is_not_a_number_stays_alone(op, n, m, what):
    """One query row of NaN or infinity: every other row of its tile as without it, and, in a step, the weights of
    the other key/value head too."""
    lay, q, kt, vt, kc, vc, table, end, run, _ = _zero_case((op, n, 64, m, 64), 460)
    clean = run()
    h, t = (m // 2, 0) if op == "step" else (1, m // 2)
    q[h, t] = what
    dirty = run()
    for a, b in zip(clean, dirty):
        assert np.isfinite(a).all()
        if op == "step":
            assert np.isnan(b[h]).all() and np.array_equal(np.delete(a, h, 0), np.delete(b, h, 0))
        else:
            assert np.isnan(b[h, t]).all()
            b[h, t] = a[h, t]
            assert np.array_equal(a, b)
    lay.close()


@pytest.mark.parametrize("op,n,m", [("step", 1000, 2), ("step", 5000, 2), ("step", 3000, 16)])
def test_weights_of_a_query_that_is_not_a_number(op, n, m):
    lay, q, kt, vt, kc, vc, table, end, run, _ = _zero_case((op, n, 64, m, 64), 470)
    w = torch.zeros((2, n), device="cuda")
    args = (kc, vc, table, _i32(end - 1), lay, 1)
    bsa.decode_weights(q[:, 0].contiguous(), *args, w)
    q[m // 2, 0] = float("nan")                       # of the first key/value head
    w2 = torch.zeros_like(w)
    bsa.decode_weights(q[:, 0].contiguous(), *args, w2)
    torch.cuda.synchronize()
    assert torch.isnan(w2[0, :end]).all() and torch.equal(w2[1], w[1]) and not torch.any(w2[:, end:])
    lay.close()


# ------------------------------------------------------------------ captured among other work

@pytest.mark.parametrize("n", [1000, 5000])
def test_captured_behind_copies_clears_and_other_streams(n):
    """One graph in which each call follows a copy, a clear, a kernel or another stream's work that writes what it
    reads, and is followed by one that changes it: replayed, the bits of the same work launched eagerly and waited for."""
    B, H, G, d, T, budget = 64, 4, 2, 64, 5, n // 3
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=n // B + 1, global_first=0))
    kc0, vc0, table, _ = _paged(1, G, n, B, d, 480)
    q0, kt0, vt0 = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, T, d, seeds=(481, 482, 483)))
    qp, kp, vp = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, n, d, seeds=(484, 485, 486)))
    _, lse_p = bsa.attention(qp, kp, vp, lay)
    par0, pos0, len0 = _i32(-1, 0, 0, 1, 3).view(1, T), _i32(n - 20), _i32(n - 19)
    h = lay.handle
    ws = [torch.empty(max(16, x), dtype=torch.uint8, device="cuda") for x in (
        bsa.bsa_attention_weights_workspace_bytes(h, H, G), bsa.bsa_decode_weights_workspace_bytes(h, 1, H, G, d),
        bsa.bsa_decode_tree_workspace_bytes(h, 1, H, G, T, d), bsa.bsa_evict_workspace_bytes(h, 1, G, budget))]

    def bufs():
        return dict(q=torch.zeros_like(q0), q1=torch.zeros_like(q0[:, 0]), kt=torch.zeros_like(kt0), vt=torch.zeros_like(vt0),
                    kc=kc0.clone(), vc=vc0.clone(), par=torch.zeros_like(par0), pos=torch.zeros_like(pos0),
                    len=torch.zeros_like(len0), w=torch.full((G, n), 3.0, device="cuda"), o=torch.zeros_like(q0),
                    lse=torch.zeros((H, T), device="cuda"), o1=torch.zeros_like(q0[:, 0]), lse1=torch.zeros(H, device="cuda"),
                    wo=torch.zeros((G, n), device="cuda"), to=torch.zeros((G, n), dtype=torch.int32, device="cuda"),
                    lo=torch.zeros_like(len0))

    def work(x, other, wait):
        main = torch.cuda.current_stream()
        x["w"].zero_()
        wait()
        bsa.attention_weights(qp, kp, lse_p, lay, x["w"], workspace=ws[0])
        wait()
        x["q1"].copy_(q0[:, 0])
        x["pos"].copy_(pos0)
        wait()
        bsa.decode_weights(x["q1"], x["kc"], x["vc"], table, x["pos"], lay, 1, x["w"], o=x["o1"], lse=x["lse1"], workspace=ws[1])
        x["q1"].zero_()
        x["w"].add_(1.0)
        wait()
        # the tree and its inputs on another stream, the cut on this one once both are done
        other.wait_stream(main)
        with torch.cuda.stream(other):
            for a, b in (("q", q0), ("kt", kt0), ("vt", vt0), ("par", par0), ("len", len0)):
                x[a].copy_(b)
            wait()
            bsa.decode_tree(x["q"], x["kt"], x["vt"], x["kc"], x["vc"], table, x["len"], x["par"], lay, o=x["o"], lse=x["lse"],
                            workspace=ws[2])
        main.wait_stream(other)
        wait()
        bsa.evict(x["kc"], x["vc"], table, x["len"], x["w"], lay, budget, 10, weights_out=x["wo"], tokens_out=x["to"],
                  lengths_out=x["lo"], workspace=ws[3])
        x["len"].zero_()
        x["w"].fill_(-1.0)

    want, got, live = bufs(), bufs(), bufs()
    other = torch.cuda.Stream()
    work(want, other, torch.cuda.synchronize)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work(got, other, lambda: None)
    for _ in range(3):
        for name in ("kc", "vc"):
            got[name].copy_({"kc": kc0, "vc": vc0}[name])
            live[name].copy_(got[name])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        work(live, other, lambda: None)
        torch.cuda.synchronize()
        for name in want:
            for x in (got, live):
                assert torch.equal(x[name].contiguous().view(torch.uint8), want[name].contiguous().view(torch.uint8)), name
    assert got["lo"].tolist() == [budget] and torch.isfinite(got["wo"]).all()
    bsa.bsa_get_status(h)
    del g
    lay.close()
