"""GPU parity of the cache operators (through the C ABI) against the fp64
oracle: the weights of a prompt's keys, the decode step that adds its weights
up, the cut of a cache by them and the attention of a drafted tree; then a
run of all of them as a server would make it.

Tolerances, derived from the kernels' arithmetic.  With q, k exact bf16 and
products summed in fp32, a score is off by at most
  e_s = scale (d + 2) 2^-24 max|q| max|k|   (2-norms; Cauchy-Schwarz)
and an exponential's argument, formed in exp2 units of magnitude at most X, by
3 roundings of 2^-24 X more; exp2 itself by 2^-22 relative.  So a probability
is off by a factor e_p = e_s + 3 ln2 2^-24 X + 2^-22.  P goes into the product
as two bf16 numbers: its upper 16 bits, which leave less than 2^-7 of P, and
that rest rounded to nearest, by at most 2^-8 of itself: 2^-15 of P in all.
  lse: e_p plus its own rounding and log2's, 2^-22 (|lse| + 1)
  o:   half a bf16 step plus 2 (e_p + 2^-15) max|v|
  w:   each term e_p plus the rounding of lse (2^-24 |lse|, the same fp32 lse
       is given to the oracle for the prompt), sums of N terms N 2^-24: with
       rows summed 32 deep per thread and at most `runs` runs joined,
       N = 32 + 8 + runs.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_sparse_long_bsa_b200 as bsa
from block_sparse_long_bsa_b200 import inputs
from oracle import cache as OC
from oracle import decode as OD
from oracle import layouts as OL

from gpu_common import bf16_half_ulp, to_device_bf16

pytestmark = pytest.mark.gpu

DYADIC = dict(window=2, global_first=1, dyadic_kmin=2)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bsa.load_library()


def _norm(x):
    return float(np.sqrt((np.nan_to_num(x) ** 2).sum(-1)).max()) if x.size else 0.0


def _e_p(scale, d, q, k, lse):
    fin = lse[np.isfinite(lse)]
    top = scale * _norm(q) * _norm(k) + (np.abs(fin).max() if fin.size else 0.0)
    return scale * (d + 2) * 2.0 ** -24 * _norm(q) * _norm(k) + 3 * 2.0 ** -24 * top + 2.0 ** -22


def _close_lse(got, want, e_p):
    fin = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fin) and np.array_equal(got[~fin], want[~fin])
    bound = e_p + 2.0 ** -22 * (np.abs(want[fin]) + 1)
    assert np.all(np.abs(got[fin] - want[fin]) <= bound), (np.abs(got[fin] - want[fin]) / bound).max()


def _close_o(got, want, e_p, v):
    bound = bf16_half_ulp(got) + 2 * (e_p + 2.0 ** -15) * float(np.abs(np.nan_to_num(v)).max())
    assert np.all(np.abs(got - want) <= bound), (np.abs(got - want) / bound).max()


def _close_w(got, want, e_p, lse, terms=80):
    fin = lse[np.isfinite(lse)]
    rel = e_p + 2.0 ** -24 * (np.abs(fin).max() if fin.size else 0) + terms * 2.0 ** -24
    bound = np.abs(want) * rel + 1e-30
    assert np.all(np.abs(got - want) <= bound), (np.abs(got - want) / bound).max()


def _np(t):
    return t.double().cpu().numpy()


def _layout(kind, n, B, L, pat):
    return bsa.Layout(kind, n, B, L, torch.cuda.current_device(), **pat)


def _mask_pattern(n, B, L, seed, keep=0.4):
    """An explicit mask with rows that keep nothing and rows without their own block."""
    nb = -(-n // B)
    m = np.tril(np.random.default_rng(seed).random((L, nb, nb)) < keep)
    m[:, ::5] = False
    return dict(mask=m.astype(np.uint8)), [[set(np.nonzero(m[h, i])[0].tolist()) for i in range(nb)] for h in range(L)]


def _sets(kind, n, B, L, pat, seed=3):
    if kind == OL.EXPLICIT:
        return _mask_pattern(n, B, L, seed)
    return pat, OL.kept_sets(kind, n, B, L, **pat)


# ------------------------------------------------------------------ weights of a prompt

PROMPT = [
    (OL.DYADIC, 1000, 64, 1, 4, 2, 128, DYADIC),
    (OL.DYADIC, 1500, 128, 1, 6, 2, 64, DYADIC),                    # three query heads a key/value head
    (OL.RANDOM, 900, 64, 4, 8, 4, 64, dict(density=0.4, seed=5)),   # a route for each query head
    (OL.RANDOM, 700, 128, 2, 4, 4, 128, dict(density=0.5, seed=6)),
    (OL.BAND_GLOBAL, 64 * 40, 64, 1, 2, 2, 64, dict(window=40, global_first=0)),   # columns of several runs
    (OL.BAND_GLOBAL, 1, 64, 1, 1, 1, 64, dict(window=0, global_first=0)),
    (OL.BAND_GLOBAL, 65, 64, 1, 3, 1, 128, dict(window=1, global_first=0)),
    (OL.EXPLICIT, 777, 64, 1, 2, 1, 64, None),
    (OL.EXPLICIT, 777, 128, 2, 4, 2, 128, None),
]


@pytest.mark.parametrize("case", PROMPT)
def test_prompt_weights(case):
    kind, n, B, L, H, G, d, pat = case
    pat, sets = _sets(kind, n, B, L, pat)
    lay = _layout(kind, n, B, L, pat)
    qb, kb, vb = inputs.qkv_bits(H, G, n, d, seeds=(1, 2, 3))
    q, k, v = (to_device_bf16(x) for x in (qb, kb, vb))
    scale = d ** -0.5
    _, lse = bsa.attention(q, k, v, lay, scale)
    start = torch.rand((G, n + 7), device="cuda")                   # a longer row, and weights from before
    w = start.clone()
    out = bsa.attention_weights(q, k, lse, lay, w[:, :n], scale)
    again = start.clone()
    bsa.attention_weights(q, k, lse, lay, again[:, :n], scale)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    assert out.data_ptr() == w.data_ptr() and torch.equal(w, again) and torch.equal(w[:, n:], start[:, n:])
    qh, kh = (inputs.bf16_bits_to_f64(x) for x in (qb, kb))
    lse_h = _np(lse)
    want = OC.prompt_weights(qh, kh, lse_h, sets, B, scale)
    got, base = _np(w[:, :n]), _np(start[:, :n])
    e_p = _e_p(scale, d, qh, kh, lse_h)
    rel = e_p + 2.0 ** -24 * np.abs(lse_h[np.isfinite(lse_h)]).max() + (40 + H * (n // (16 * B) + 1)) * 2.0 ** -24
    bound = want * rel + 2.0 ** -24 * (want + base)                 # the addition to what was there
    assert np.all(np.abs(got - base - want) <= bound), (np.abs(got - base - want) / bound).max()
    lay.close()


def test_prompt_weights_in_strips():
    """So many kept blocks that key/value heads take the workspace in turns: some columns against fp64, all by
    their total (every query row gives one)."""
    n, B, H, G, d = 64 * 600, 64, 8, 4, 64
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=n // B, global_first=0))
    assert (600 * 601 // 2) * B * 4 > (64 << 20) // 2               # one key/value head at a time
    q, k, v = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, n, d, seeds=(7, 8, 9)))
    _, lse = bsa.attention(q, k, v, lay)
    w, w2 = bsa.attention_weights(q, k, lse, lay), bsa.attention_weights(q, k, lse, lay)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    assert torch.equal(w, w2)
    # a score is off by e_s <= 2e-5 here (norms up to 11), a row's sum of terms by no more, and lse by 2^-23 of it
    assert float((w.double().sum(1) / n - H // G).abs().max()) <= H // G * 3e-5
    for u in (0, 5, 63, 64, 19200, 30001, n - 1):
        x = (q[:, u:].double() * k.repeat_interleave(2, 0)[:, u:u + 1].double()).sum(-1) * d ** -0.5
        want = torch.exp(x - lse[:, u:].double()).sum(-1).view(G, 2).sum(1)
        assert float(((w[:, u].double() - want) / want).abs().max()) <= 3e-5
    lay.close()


def test_prompt_weights_of_rows_that_are_not_numbers_stay_in_their_columns():
    """A NaN or infinite query row reaches only the keys it may read; rows with lse = -inf give nothing;
    a NaN key only its own column."""
    n, B, d = 500, 64, 64
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=1, global_first=0))
    sets = OL.kept_sets(OL.BAND_GLOBAL, n, B, 1, window=1, global_first=0)
    qb, kb, vb = inputs.qkv_bits(2, 1, n, d, seeds=(4, 5, 6))
    q, k, v = (to_device_bf16(x) for x in (qb, kb, vb))
    _, lse = bsa.attention(q, k, v, lay)
    q[0, 200] = float("nan")                # block 3, reads 128 .. 200
    q[1, 310] = float("inf")                # block 4, reads 192 .. 310
    k[0, 450] = float("nan")                # read by rows 450 .. 499
    lse = lse.clone()
    lse[:, 100:120] = float("-inf")
    w = bsa.attention_weights(q, k, lse, lay)
    torch.cuda.synchronize()
    got, qh, kh = _np(w), _np(q), _np(k)
    touched = np.zeros(n, bool)
    touched[128:201] = touched[192:311] = touched[450] = True
    want = OC.prompt_weights(np.nan_to_num(qh, posinf=0, neginf=0), np.nan_to_num(kh), _np(lse), sets, B, d ** -0.5)
    assert np.isnan(got[0, 128:201]).all() and np.isnan(got[0, 450])
    assert np.isfinite(got[0, ~touched]).all()
    rel = 2e-5                              # far above the bound of the test above, far below a missing row
    assert np.all(np.abs(got[0, ~touched] - want[0, ~touched]) <= rel * want[0, ~touched] + 1e-6)
    lay.close()


@pytest.mark.parametrize("B,H", [(64, 1), (64, 2), (128, 1)])
def test_prompt_weights_of_a_key_that_no_row_gives_weight(B, H):
    """A key at minus infinity for every row that reads it gets a weight of 0, in a last block that the sequence
    does not fill too: the block's rows past the end have no say."""
    n, d = 450, 64
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=1, global_first=0))
    sets = OL.kept_sets(OL.BAND_GLOBAL, n, B, 1, window=1, global_first=0)
    qb, kb, vb = inputs.qkv_bits(H, 1, n, d, seeds=(14, 15, 16))
    q, k, v = (to_device_bf16(x) for x in (qb, kb, vb))
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    k[0, [100, 380, 400, 449], 0] = float("-inf")
    _, lse = bsa.attention(q, k, v, lay)
    lse_h = _np(lse)
    assert np.isfinite(lse_h).all()
    w = bsa.attention_weights(q, k, lse, lay)
    torch.cuda.synchronize()
    got = _np(w)
    want = OC.prompt_weights(_np(q), _np(k), lse_h, sets, B, d ** -0.5)
    e_p = _e_p(d ** -0.5, d, _np(q), np.nan_to_num(_np(k), neginf=0), lse_h)
    assert (want[0, [100, 380, 400, 449]] == 0).all()
    _close_w(got, want, e_p, lse_h)
    lay.close()


# ------------------------------------------------------------------ paged caches

def _paged(batch, G, n, B, d, seed, spare=0):
    """Keys and values as contiguous fp64 and as a shuffled paged cache on the GPU whose unused rows are NaN."""
    _, kb, vb = inputs.qkv_bits(1, batch * G, n, d, seeds=(seed, seed + 1, seed + 2))
    nb = -(-n // B)
    order = np.random.default_rng(seed).permutation(batch * nb + spare)[:batch * nb]
    table = order.reshape(batch, nb).astype(np.int32)
    kc = torch.full((batch * nb + spare, G, B, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    for c, bits in ((kc, kb), (vc, vb)):
        x = to_device_bf16(bits).view(batch, G, n, d)
        pad = torch.full((batch, G, nb * B, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        pad[:, :, :n] = x
        c[torch.from_numpy(table.astype(np.int64)).cuda()] = pad.view(batch, G, nb, B, d).transpose(1, 2)
    return kc, vc, torch.from_numpy(table).cuda(), table


def _blank(kc, vc, table, B, lengths):
    """NaN in every cached row at or past a sequence's length."""
    for b, m in enumerate(lengths):
        for j in range(table.shape[1]):
            lo = min(max(m - j * B, 0), B)
            kc[int(table[b, j]), :, lo:] = float("nan")
            vc[int(table[b, j]), :, lo:] = float("nan")


STEP = [
    (OL.DYADIC, 3000, 64, 1, 2, 4, 2, 128, DYADIC),
    (OL.RANDOM, 3000, 128, 4, 2, 4, 4, 128, dict(density=0.3, seed=4)),
    (OL.RANDOM, 1500, 64, 6, 2, 6, 2, 64, dict(density=0.3, seed=9)),   # routes differ inside a group
    (OL.BAND_GLOBAL, 1000, 64, 1, 3, 2, 1, 64, dict(window=2, global_first=1)),
    (OL.BAND_GLOBAL, 2500, 128, 1, 1, 40, 1, 64, dict(window=20, global_first=0)),   # 40 query heads a key/value head
    (OL.BAND_GLOBAL, 700, 64, 1, 1, 130, 1, 128, dict(window=11, global_first=0)),   # more than one tile of them
    (OL.EXPLICIT, 1100, 64, 1, 2, 2, 2, 64, None),
    (OL.EXPLICIT, 1100, 128, 4, 2, 4, 2, 128, None),
]


@pytest.mark.parametrize("case", STEP)
def test_step_weights(case):
    kind, n, B, L, batch, H, G, d, pat = case
    pat, sets = _sets(kind, n, B, L, pat)
    lay = _layout(kind, n, B, L, pat)
    scale = d ** -0.5
    rng = np.random.default_rng(7)
    for at in ([0] * batch, [B - 1] * batch, [B] * batch, [n - 1] * batch, [int(x) for x in rng.integers(0, n, batch)]):
        kc, vc, table, th = _paged(batch, G, n, B, d, 20)
        _blank(kc, vc, th, B, [t + 1 for t in at])
        qb = inputs.normal_bf16_bits((batch * H, d), 30)
        q, qh = to_device_bf16(qb), inputs.bf16_bits_to_f64(qb)
        pos = torch.tensor(at, dtype=torch.int32, device="cuda")
        start = torch.rand((batch * G, n + 5), device="cuda")
        w = start.clone()
        o, lse = bsa.decode_weights(q, kc, vc, table, pos, lay, batch, w, scale)
        w2 = start.clone()
        o2, lse2 = bsa.decode_weights(q, kc, vc, table, pos, lay, batch, w2, scale)
        torch.cuda.synchronize()
        bsa.bsa_get_status(lay.handle)
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(w, w2)
        kh, vh = np.nan_to_num(_np(kc)), np.nan_to_num(_np(vc))
        o_ref, lse_ref = OD.decode_step(qh, kh, vh, th, at, sets, B, scale)
        e_p = _e_p(scale, d, qh, kh, lse_ref)
        _close_lse(_np(lse), lse_ref, e_p)
        _close_o(_np(o), o_ref, e_p, vh)
        want = OC.step_weights(qh, kh, th, at, lse_ref, sets, B, scale, n)
        got, base = _np(w), _np(start)
        assert np.array_equal(got[:, n:], base[:, n:])
        bound = want * (2 * e_p + 2.0 ** -21 + (H // G) * 2.0 ** -24) + 2.0 ** -24 * (want + base[:, :n])
        diff = np.abs(got[:, :n] - base[:, :n] - want)
        assert np.all(diff <= bound), (diff / bound).max()
        assert np.array_equal(got[:, :n][want == 0], base[:, :n][want == 0])
    lay.close()


@pytest.mark.parametrize("H,G,d,B", [(16, 16, 64, 64), (48, 16, 64, 128), (128, 16, 64, 64), (64, 8, 128, 64), (128, 8, 64, 64)])
@pytest.mark.parametrize("late", [False, True])
def test_step_whose_maxima_keep_moving(H, G, d, B, late):
    """1 to 16 query heads a key/value head over runs of several chunks: scores that rise by 10 from chunk to chunk
    (even heads) or fall (odd heads), and, `late`, no finite score in the first 192 tokens."""
    n, batch = 1000, 128 // G
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=-(-n // B), global_first=0))
    sets = OL.kept_sets(OL.BAND_GLOBAL, n, B, 1, window=-(-n // B), global_first=0)
    kc, vc, table, th = _paged(batch, G, n, B, d, 50)
    at = [n - 1 - 37 * b for b in range(batch)]
    token = torch.arange(-(-n // B) * B, device="cuda").view(-1, B)
    for b in range(batch):
        pages = table[b].long()
        kc[pages] *= 0.25
        kc[pages, :, :, 0] = (token // 64 * 10).to(torch.bfloat16)[:, None]
        if late:
            kc[pages, :, :, 1] = torch.where(token < 192, float("-inf"), 0.5).to(torch.bfloat16)[:, None]
    _blank(kc, vc, th, B, [t + 1 for t in at])
    q = to_device_bf16(inputs.normal_bf16_bits((batch * H, d), 51)) * 0.25
    q[:, 0] = torch.where(torch.arange(batch * H, device="cuda") % 2 == 0, 1.0, -1.0)
    q[:, 1] = 0.5
    w = torch.zeros((batch * G, n), device="cuda")
    o, lse = bsa.decode_weights(q, kc, vc, table, torch.tensor(at, dtype=torch.int32, device="cuda"), lay, batch, w, 1.0)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    qh, kh, vh = _np(q), np.nan_to_num(_np(kc), neginf=-np.inf), np.nan_to_num(_np(vc))
    o_ref, lse_ref = OD.decode_step(qh, kh, vh, th, at, sets, B, 1.0)
    e_p = _e_p(1.0, d, qh, np.where(np.isinf(kh), 0, kh), lse_ref)
    _close_lse(_np(lse), lse_ref, e_p)
    _close_o(_np(o), o_ref, e_p, vh)
    want = OC.step_weights(qh, kh, th, at, lse_ref, sets, B, 1.0, n)
    bound = want * (2 * e_p + 2.0 ** -21 + (H // G) * 2.0 ** -24) + 1e-30
    assert np.all(np.abs(_np(w) - want) <= bound), (np.abs(_np(w) - want) / bound).max()
    assert e_p < 5e-3 and (not late or (want[:, :192] == 0).all())
    lay.close()


def test_step_agrees_with_decode_and_long_rows_split():
    n, B, batch, H, G, d = 32768, 64, 2, 4, 2, 128
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=n // B, global_first=0))
    kc, vc, table, _ = _paged(batch, G, n, B, d, 40)
    q = to_device_bf16(inputs.normal_bf16_bits((batch * H, d), 41))
    pos = torch.tensor([n - 1, 12345], dtype=torch.int32, device="cuda")
    w = torch.zeros((batch * G, n), device="cuda")
    o, lse = bsa.decode_weights(q, kc, vc, table, pos, lay, batch, w)
    o2, lse2 = bsa.decode(q, kc, vc, table, pos, lay, batch)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    # each is within half a bf16 step and 2e-4 (e_p of 9e-5 at these sizes) of the same number
    bound = bf16_half_ulp(_np(o)) + bf16_half_ulp(_np(o2)) + 8e-4
    assert np.all(np.abs(_np(o) - _np(o2)) <= bound)
    assert float((lse - lse2).abs().max()) <= 2e-4
    # every query row gives one in all: terms are off by e_p each, the sum of 32768 of them by no more
    got = w.double().sum(1)
    assert float((got - H // G).abs().max()) <= 2 * (H // G) * 2e-4
    assert torch.all(w[G:, 12346:] == 0)
    lay.close()


def test_step_refuses_bad_indices_on_the_device():
    n, B, batch, H, G, d = 1024, 64, 3, 4, 2, 64
    lay = _layout(OL.DYADIC, n, B, 1, DYADIC)
    kc, vc, table, th = _paged(batch, G, n, B, d, 50, spare=2)
    q = to_device_bf16(inputs.normal_bf16_bits((batch * H, d), 51))
    good = torch.tensor([500, 700, 900], dtype=torch.int32, device="cuda")
    w0 = torch.rand((batch * G, n), device="cuda")
    ref = w0.clone()
    o_ref, lse_ref = bsa.decode_weights(q, kc, vc, table, good, lay, batch, ref)
    for pos, tab in ((torch.tensor([-1, 700, n], dtype=torch.int32, device="cuda"), table), (good, table.clone())):
        if tab is not table:
            tab[0, 500 // B] = -1
            tab[2, 0] = kc.shape[0]
        w = w0.clone()
        o, lse = bsa.decode_weights(q, kc, vc, tab, pos, lay, batch, w)
        torch.cuda.synchronize()
        with pytest.raises(bsa.BsaError):
            bsa.bsa_get_status(lay.handle)
        bsa.bsa_get_status(lay.handle)
        for b in (0, 2):
            assert torch.all(o[b * H:(b + 1) * H] == 0) and torch.all(torch.isneginf(lse[b * H:(b + 1) * H]))
            assert torch.equal(w[b * G:(b + 1) * G], w0[b * G:(b + 1) * G])
        assert torch.equal(o[H:2 * H], o_ref[H:2 * H]) and torch.equal(w[G:2 * G], ref[G:2 * G])
        assert torch.equal(lse[H:2 * H], lse_ref[H:2 * H])
    lay.close()


# ------------------------------------------------------------------ the cut

EVICT = [
    # n, B, batch, G, d, budget, recent, lengths, ids
    (300, 64, 2, 2, 64, 100, 10, [300, 177], False),
    (300, 128, 3, 1, 128, 100, 0, [100, 99, 101], True),
    (1000, 64, 2, 3, 128, 1, 1, [1000, 0], True),
    (1000, 64, 2, 2, 64, 999, 999, [1000, 1], True),
    (2500, 128, 1, 2, 64, 2400, 300, [2500], True),
    (5000, 64, 2, 1, 128, 64, 32, [4999, 65], False),
    (64, 64, 1, 1, 64, 100, 3, [64], False),                # a budget past the cache: nothing to cut
    (70000, 128, 1, 1, 64, 30001, 500, [69999], True),      # a cluster of blocks for each row
    (400000, 128, 1, 1, 64, 100001, 500, [399999], True),   # longer than the keys that their shared memory holds
    (1024, 128, 2, 2, 64, 512, 64, [1024, 700], False),     # few slots: one kernel
    (1025, 64, 2, 2, 128, 512, 64, [1025, 513], True),      # two
    (3000, 64, 3, 2, 128, 2950, 100, [3000, 2960, 10], True),   # few moves: one
    (4096, 64, 2, 2, 64, 1500, 0, [4096, 1501], False),     # two
]


def _cut_case(case, weights=None):
    n, B, batch, G, d, budget, recent, lengths, ids = case
    rng = np.random.default_rng(60)
    kc, vc, table, th = _paged(batch, G, n, B, d, 61)
    if weights is None:
        w = np.round(np.exp(2 * rng.standard_normal((batch * G, n))), 1).astype(np.float32)   # ties, zeros among them
    else:
        w = weights(rng, batch * G, n)
    tok = (2 * np.stack([rng.permutation(n) for _ in range(batch * G)])).astype(np.int32) if ids else None
    return kc, vc, table, th, w, tok


def _run_cut(lay, case, kc, vc, table, w, tok):
    n, B, batch, G, d, budget, recent, lengths, ids = case
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    t = torch.from_numpy(tok).cuda() if tok is not None else None
    return bsa.evict(kc, vc, table, lens, torch.from_numpy(w).cuda(), lay, budget, recent, tokens=t)


def _check_cut(case, before, after, out, th, w, tok):
    n, B, batch, G, d, budget, recent, lengths, ids = case
    kh, vh, w_ref, t_ref, l_ref = OC.evict(before[0], before[1], th, lengths, w, tok, n, budget, recent)
    np.testing.assert_array_equal(after[0], kh)
    np.testing.assert_array_equal(after[1], vh)
    np.testing.assert_array_equal(out[0].cpu().numpy(), w_ref)
    np.testing.assert_array_equal(out[1].cpu().numpy(), t_ref)
    np.testing.assert_array_equal(out[2].cpu().numpy(), l_ref)


@pytest.mark.parametrize("case", EVICT)
def test_evict(case):
    n, B, batch, G, d, budget, recent, lengths, ids = case
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=0, global_first=0))
    kc, vc, table, th, w, tok = _cut_case(case)
    before = (_np(kc), _np(vc))
    out = _run_cut(lay, case, kc, vc, table, w, tok)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    _check_cut(case, before, (_np(kc), _np(vc)), out, th, w, tok)
    lay.close()


@pytest.mark.parametrize("kind", ["equal", "zero", "special", "negative", "close"])
def test_evict_order_of_weights(kind):
    """All equal (the lowest slots stay), zeros of both signs, NaN and infinities, negative ones, and neighbours
    in the last bit."""
    def weights(rng, rows, n):
        if kind == "equal":
            return np.full((rows, n), 3.25, np.float32)
        if kind == "zero":
            return np.where(rng.random((rows, n)) < 0.5, np.float32(0.0), np.float32(-0.0)).astype(np.float32)
        if kind == "special":
            return rng.choice(np.array([np.nan, np.inf, -np.inf, 0, 1, 1e-45, 3e38, -1], np.float32), (rows, n))
        if kind == "negative":
            return rng.standard_normal((rows, n)).astype(np.float32)
        return (np.float32(1) + rng.integers(0, 50, (rows, n)) * np.float32(2.0 ** -23)).astype(np.float32)
    for budget in (1, 500, 1400):
        case = (1500, 64, 2, 2, 64, budget, 0, [1500, 1111], False)
        lay = _layout(OL.BAND_GLOBAL, 1500, 64, 1, dict(window=0, global_first=0))
        kc, vc, table, th, w, tok = _cut_case(case, weights)
        before = (_np(kc), _np(vc))
        out = _run_cut(lay, case, kc, vc, table, w, tok)
        torch.cuda.synchronize()
        bsa.bsa_get_status(lay.handle)
        _check_cut(case, before, (_np(kc), _np(vc)), out, th, w, tok)
        lay.close()


def test_evict_leaves_a_refused_sequence_as_it_was():
    n, B, batch, G, d, budget = 640, 64, 4, 2, 64, 100
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=0, global_first=0))
    case = (n, B, batch, G, d, budget, 5, [n + 1, 300, -1, 300], False)
    kc, vc, table, th, w, tok = _cut_case(case)
    bad = table.clone()
    bad[1, 2] = kc.shape[0]                     # a page that does not exist, among the sequence's tokens
    bad[3, 5] = -7                              # one past them: never looked at
    before = (_np(kc), _np(vc))
    w_out = torch.full((batch * G, n), 7.0, device="cuda")
    t_out = torch.full((batch * G, n), 7, dtype=torch.int32, device="cuda")
    lens = torch.tensor([n + 1, 300, -1, 300], dtype=torch.int32, device="cuda")
    _, _, l_out = bsa.evict(kc, vc, bad, lens, torch.from_numpy(w).cuda(), lay, budget, 5, weights_out=w_out,
                            tokens_out=t_out)
    torch.cuda.synchronize()
    with pytest.raises(bsa.BsaError):
        bsa.bsa_get_status(lay.handle)
    assert l_out.tolist() == [-1, -1, -1, budget]
    assert torch.all(w_out[:6] == 7) and torch.all(t_out[:6] == 7)
    kh, vh, w_ref, t_ref, _ = OC.evict(before[0], before[1], th, [0, 0, 0, 300], w, None, n, budget, 5)
    np.testing.assert_array_equal(_np(kc), kh)
    np.testing.assert_array_equal(_np(vc), vh)
    np.testing.assert_array_equal(w_out[6:].cpu().numpy(), w_ref[6:])
    np.testing.assert_array_equal(t_out[6:].cpu().numpy(), t_ref[6:])
    lay.close()


# ------------------------------------------------------------------ the drafted tree

def _tree_parents(rng, batch, T, chain):
    par = np.full((batch, T), -2, np.int32)
    for b in range(batch):
        for i in range(T if b == 0 else max(1, T - b)):
            par[b, i] = i - 1 if rng.random() < chain else rng.integers(-1, i) if i else -1
    return par


TREE = [
    # kind, n, B, L, batch, H, G, d, pat, T, chain, lengths
    (OL.DYADIC, 3000, 64, 1, 2, 4, 2, 128, DYADIC, 7, 0.3, [2500, 63]),
    (OL.DYADIC, 3000, 64, 1, 2, 4, 2, 128, DYADIC, 1, 0.3, [2999, 64]),
    (OL.DYADIC, 3000, 64, 1, 2, 8, 2, 64, DYADIC, 128, 1.0, [2600, 127]),        # chains over three layout rows
    (OL.DYADIC, 2000, 128, 1, 1, 2, 2, 128, DYADIC, 128, 0.9, [1000]),
    (OL.RANDOM, 3000, 128, 4, 2, 4, 4, 128, dict(density=0.3, seed=4), 9, 0.7, [2687, 0]),
    (OL.RANDOM, 1500, 64, 6, 2, 6, 2, 64, dict(density=0.3, seed=9), 33, 0.7, [1000, 31]),
    (OL.BAND_GLOBAL, 1000, 64, 1, 3, 3, 1, 64, dict(window=2, global_first=1), 64, 0.0, [900, 60, 1]),
    (OL.BAND_GLOBAL, 1000, 64, 1, 1, 16, 1, 128, dict(window=16, global_first=0), 100, 0.5, [801]),   # 1600 rows
    (OL.EXPLICIT, 1100, 64, 1, 2, 2, 2, 64, None, 20, 0.8, [310, 640]),
    (OL.EXPLICIT, 1100, 128, 4, 2, 4, 2, 128, None, 40, 0.8, [630, 250]),
]


@pytest.mark.parametrize("case", TREE)
def test_tree(case):
    kind, n, B, L, batch, H, G, d, pat, T, chain, lengths = case
    pat, sets = _sets(kind, n, B, L, pat)
    lay = _layout(kind, n, B, L, pat)
    scale = d ** -0.5
    par = _tree_parents(np.random.default_rng(T), batch, T, chain)
    kc, vc, table, th = _paged(batch, G, n, B, d, 70)
    _blank(kc, vc, th, B, lengths)
    qb, ktb, vtb = inputs.qkv_bits(batch * H, batch * G, T, d, seeds=(71, 72, 73))
    q, kt, vt = (to_device_bf16(x) for x in (qb, ktb, vtb))
    args = (q, kt, vt, kc, vc, table, torch.tensor(lengths, dtype=torch.int32, device="cuda"),
            torch.from_numpy(par).cuda(), lay, scale)
    o0 = torch.full((batch * H, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse0 = torch.full((batch * H, T), 7.0, device="cuda")
    o, lse = bsa.decode_tree(*args, o=o0, lse=lse0)
    o2, lse2 = bsa.decode_tree(*args, o=torch.full_like(o0, 7.0), lse=torch.full_like(lse0, 7.0))
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    qh, kth, vth = (inputs.bf16_bits_to_f64(x) for x in (qb, ktb, vtb))
    kh, vh = np.nan_to_num(_np(kc)), np.nan_to_num(_np(vc))
    o_ref, lse_ref = OC.tree(qh, kth, vth, kh, vh, th, lengths, par, sets, B, scale)
    used = np.repeat(par != -2, H, axis=0)
    assert np.all(_np(o)[~used] == 7) and np.all(_np(lse)[~used] == 7)
    e_p = _e_p(scale, d, qh, np.concatenate([kh.reshape(-1, d), kth.reshape(-1, d)]), lse_ref[used])
    _close_lse(_np(lse)[used], lse_ref[used], e_p)
    _close_o(_np(o)[used], o_ref[used], e_p, np.concatenate([vh.reshape(-1, d), vth.reshape(-1, d)]))
    lay.close()


def test_tree_branches_and_routes_never_meet():
    """A NaN or infinite key or value reaches the rows that read it and no others: of another branch, of a block
    that the row's layout row drops, or behind the cached tokens."""
    n, B, H, G, d, T = 1024, 64, 2, 1, 64, 6
    m = np.tril(np.ones((16, 16), np.uint8))[None]
    m[0, 8, 3] = 0                           # row 8 drops block 3, row 7 keeps it
    lay = bsa.Layout(OL.EXPLICIT, n, B, 1, torch.cuda.current_device(), mask=m)
    kc, vc, table, th = _paged(1, G, n, B, d, 80)
    length = 8 * B - 2                       # depths 0, 1 in block 7, deeper ones in block 8
    _blank(kc, vc, th, B, [length])
    par = torch.tensor([[-1, 0, 1, 2, -1, 4]], dtype=torch.int32, device="cuda")
    q, kt, vt = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, T, d, seeds=(81, 82, 83)))
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")

    def run():
        o, lse = bsa.decode_tree(q, kt, vt, kc, vc, table, lens, par, lay)
        torch.cuda.synchronize()
        return o.clone(), lse.clone()

    o, lse = run()
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
    kt[0, 5], vt[0, 5] = float("nan"), float("inf")           # the leaf of the second branch
    o2, lse2 = run()
    assert torch.equal(o2[:, :5], o[:, :5]) and torch.equal(lse2[:, :5], lse[:, :5])
    assert torch.isnan(lse2[:, 5]).all()
    vc[int(th[0, 3]), 0, 10] = float("inf")                   # block 3: rows 0, 1, 4, 5 read it, rows 2, 3 do not
    o3, lse3 = run()
    assert torch.equal(o3[:, 2:4], o[:, 2:4]) and torch.equal(lse3[:, 2:4], lse[:, 2:4])
    assert torch.isinf(o3[:, [0, 1, 4]].float()).all() and torch.equal(lse3[:, [0, 1, 4]], lse[:, [0, 1, 4]])
    bsa.bsa_get_status(lay.handle)
    lay.close()


def test_tree_refuses_bad_indices_on_the_device():
    n, B, batch, H, G, d, T = 640, 64, 4, 2, 2, 64, 8
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=10, global_first=0))
    kc, vc, table, th = _paged(batch, G, n, B, d, 90, spare=1)
    q, kt, vt = (to_device_bf16(x) for x in inputs.qkv_bits(batch * H, batch * G, T, d, seeds=(91, 92, 93)))
    par = torch.tensor([[-1, 0, 1, 2, 3, 4, 5, 6]] * batch, dtype=torch.int32, device="cuda")
    lens = torch.tensor([100, 200, 300, 632], dtype=torch.int32, device="cuda")
    o_ref, lse_ref = bsa.decode_tree(q, kt, vt, kc, vc, table, lens, par, lay)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    par2, lens2, tab2 = par.clone(), lens.clone(), table.clone()
    lens2[0] = n + 1                         # a sequence longer than the layout
    par2[1] = torch.tensor([-1, 0, 2, 2, 7, -3, 5, 1], dtype=torch.int32)   # itself, a later token, no such name
    par2[1, 7] = 1
    tab2[2, 1] = -1                          # a page that does not exist
    lens2[3] = 635                           # the last tokens pass the layout's end
    o, lse = bsa.decode_tree(q, kt, vt, kc, vc, tab2, lens2, par2, lay)
    torch.cuda.synchronize()
    with pytest.raises(bsa.BsaError):
        bsa.bsa_get_status(lay.handle)
    bsa.bsa_get_status(lay.handle)

    def refused(b, i):
        rows = slice(b * H, (b + 1) * H)
        return bool(torch.all(o[rows, i] == 0)) and bool(torch.all(torch.isneginf(lse[rows, i])))

    assert all(refused(0, i) and refused(2, i) for i in range(T))
    assert [refused(1, i) for i in range(T)] == [False, False, True, True, True, True, True, False]
    assert torch.equal(o[H:2 * H, :2], o_ref[H:2 * H, :2])
    assert [refused(3, i) for i in range(T)] == [False] * 5 + [True] * 3
    # parents that are unused, and a length below zero
    par3, lens3 = par.clone(), lens.clone()
    par3[0, 2] = -2
    lens3[1] = -1
    o, lse = bsa.decode_tree(q, kt, vt, kc, vc, table, lens3, par3, lay, o=torch.full_like(o_ref, 7.0),
                             lse=torch.full_like(lse_ref, 7.0))
    torch.cuda.synchronize()
    with pytest.raises(bsa.BsaError):
        bsa.bsa_get_status(lay.handle)
    assert torch.all(o[:H, 2] == 7) and torch.all(lse[:H, 2] == 7)
    assert [refused(0, i) for i in range(T)] == [False, False, False] + [True] * 5
    assert all(refused(1, i) for i in range(T))
    assert torch.equal(o[2 * H:], o_ref[2 * H:]) and torch.equal(lse[2 * H:], lse_ref[2 * H:])
    lay.close()


def test_tree_row_is_the_decode_step_of_its_path():
    """Through the framework alone: a drafted chain written into the cache and decoded token by token."""
    n, B, H, G, d, T = 2048, 64, 4, 2, 128, 10
    lay = _layout(OL.DYADIC, n, B, 1, DYADIC)
    kc, vc, table, th = _paged(1, G, n, B, d, 100)
    length = 1020                            # the chain crosses into the next block
    q, kt, vt = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, T, d, seeds=(101, 102, 103)))
    par = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda")[None]
    o, lse = bsa.decode_tree(q, kt, vt, kc, vc, table, torch.tensor([length], dtype=torch.int32, device="cuda"), par, lay)
    for i in range(T):
        t = length + i
        kc[int(th[0, t // B]), :, t % B], vc[int(th[0, t // B]), :, t % B] = kt[:, i], vt[:, i]
        od, lsed = bsa.decode(q[:, i].contiguous(), kc, vc, table, torch.tensor([t], dtype=torch.int32, device="cuda"),
                              lay, 1)
        torch.cuda.synchronize()
        bound = bf16_half_ulp(_np(o[:, i])) + bf16_half_ulp(_np(od)) + 8e-4
        assert np.all(np.abs(_np(o[:, i]) - _np(od)) <= bound)
        assert float((lse[:, i] - lsed).abs().max()) <= 2e-4
    bsa.bsa_get_status(lay.handle)
    lay.close()


# ------------------------------------------------------------------ caches past 2^31 elements, shared pages

def test_caches_whose_offsets_pass_32_bits():
    """Step, tree and cut on pages at the far end of caches of 2.3e9 elements: the bits they give on small ones."""
    n, B, batch, H, G, d, T = 1000, 64, 2, 4, 4, 128, 5
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GB of device memory")
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=16, global_first=0))
    kc, vc, table, th = _paged(batch, G, n, B, d, 210)
    pages, far = kc.shape[0], 70000
    assert far * G * B * d > 2 ** 31
    big = [torch.empty((far, G, B, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for b, c in zip(big, (kc, vc)):
        b[far - pages:] = c
    table2 = table + (far - pages)
    q, kt, vt = (to_device_bf16(x) for x in inputs.qkv_bits(batch * H, batch * G, T, d, seeds=(211, 212, 213)))
    lens = torch.tensor([900, 640], dtype=torch.int32, device="cuda")
    par = torch.tensor([[-1, 0, 0, 1, 3]] * batch, dtype=torch.int32, device="cuda")
    got = []
    for k, v, t in ((kc, vc, table), (big[0], big[1], table2)):
        w = torch.zeros((batch * G, n), device="cuda")
        tree = bsa.decode_tree(q, kt, vt, k, v, t, lens, par, lay)
        step = bsa.decode_weights(q[:, 0].contiguous(), k, v, t, lens - 1, lay, batch, w)
        cut = bsa.evict(k, v, t, lens, w, lay, 300, 10)
        torch.cuda.synchronize()
        got.append([*tree, *step, w, *cut, k[-pages:].clone(), v[-pages:].clone()])
    bsa.bsa_get_status(lay.handle)
    for a, b in zip(*got):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    lay.close()


def test_sequences_that_share_their_first_pages():
    """A prefix that two sequences hold in the same pages: each gives what it gives with pages of its own."""
    n, B, H, G, d, T = 640, 64, 4, 2, 64, 6
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=10, global_first=0))
    kc, vc, table, th = _paged(2, G, n, B, d, 220)
    for c in (kc, vc):
        c[table[1, :4].long()] = c[table[0, :4].long()]
    shared = table.clone()
    shared[1, :4] = table[0, :4]
    q, kt, vt = (to_device_bf16(x) for x in inputs.qkv_bits(2 * H, 2 * G, T, d, seeds=(221, 222, 223)))
    lens = torch.tensor([500, 300], dtype=torch.int32, device="cuda")
    par = torch.tensor([[-1, 0, 1, 1, -1, 4]] * 2, dtype=torch.int32, device="cuda")
    out = []
    for t in (table, shared):
        w = torch.zeros((2 * G, n), device="cuda")
        out.append([*bsa.decode_tree(q, kt, vt, kc, vc, t, lens, par, lay),
                    *bsa.decode_weights(q[:, 0].contiguous(), kc, vc, t, lens - 1, lay, 2, w), w])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*out))
    lay.close()


@pytest.mark.parametrize("d", [64, 128])
def test_a_tree_that_straddles_blocks_of_a_whole_cache(d):
    """Where every block is kept, rows of two or three layout rows share their runs: against the oracle, with the
    cache ending at, before and behind a block's border."""
    n, B, H, G, T = 500, 64, 4, 2, 90
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=8, global_first=0))
    sets = OL.kept_sets(OL.BAND_GLOBAL, n, B, 1, window=8, global_first=0)
    par = np.array([list(range(-1, T - 1))], np.int32)
    par[0, 70:] = 20
    for length in (191, 192, 193, 250, 0):
        kc, vc, table, th = _paged(1, G, n, B, d, 230)
        _blank(kc, vc, th, B, [length])
        q, kt, vt = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, T, d, seeds=(231, 232, 233)))
        o, lse = bsa.decode_tree(q, kt, vt, kc, vc, table, torch.tensor([length], dtype=torch.int32, device="cuda"),
                                 torch.from_numpy(par).cuda(), lay)
        torch.cuda.synchronize()
        bsa.bsa_get_status(lay.handle)
        kh, vh = np.nan_to_num(_np(kc)), np.nan_to_num(_np(vc))
        o_ref, lse_ref = OC.tree(_np(q), _np(kt), _np(vt), kh, vh, th, [length], par, sets, B, d ** -0.5)
        e_p = _e_p(d ** -0.5, d, _np(q), np.concatenate([kh.reshape(-1, d), _np(kt).reshape(-1, d)]), lse_ref)
        _close_lse(_np(lse), lse_ref, e_p)
        _close_o(_np(o), o_ref, e_p, np.concatenate([vh.reshape(-1, d), _np(vt).reshape(-1, d)]))
    lay.close()


# ------------------------------------------------------------------ how they are called

def _small_tree(seed, stream=None):
    n, B, H, G, d, T = 1000, 64, 4, 2, 64, 5
    lay = _layout(OL.DYADIC, n, B, 1, DYADIC)
    kc, vc, table, th = _paged(1, G, n, B, d, seed)
    q, kt, vt = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, T, d, seeds=(seed, seed + 1, seed + 2)))
    lens = torch.tensor([900], dtype=torch.int32, device="cuda")
    par = torch.tensor([[-1, 0, 0, 1, 3]], dtype=torch.int32, device="cuda")
    return lay, q, kt, vt, kc, vc, table, lens, par


def test_calls_on_two_streams_at_once_and_in_a_graph():
    """Step, tree, cut and prompt weights on two streams at the same time, each with its own workspace, and
    captured together and replayed on new inputs: the same bits as one call after the other."""
    n, B, H, G, d, T = 1000, 64, 4, 2, 64, 5
    lay, q, kt, vt, kc, vc, table, lens, par = _small_tree(110)
    qp, kp, vp = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, n, d, seeds=(120, 121, 122)))
    op, lsep = bsa.attention(qp, kp, vp, lay)
    q1 = q[:, 0].contiguous()
    pos = torch.tensor([899], dtype=torch.int32, device="cuda")
    w0 = torch.rand((G, n), device="cuda")

    class Out:
        pass

    def bufs():
        x = Out()
        x.o, x.lse = torch.zeros_like(q), torch.zeros((H, T), device="cuda")
        x.o1, x.lse1 = torch.zeros_like(q1), torch.zeros(H, device="cuda")
        x.w, x.wp = w0.clone(), torch.zeros((G, n), device="cuda")
        x.kc, x.vc = kc.clone(), vc.clone()
        x.wo, x.to, x.lo = torch.zeros((G, n), device="cuda"), torch.zeros((G, n), dtype=torch.int32, device="cuda"), lens.clone()
        h = lay.handle
        x.ws = [torch.empty(max(16, s), dtype=torch.uint8, device="cuda") for s in (
            bsa.bsa_decode_tree_workspace_bytes(h, 1, H, G, T, d), bsa.bsa_decode_weights_workspace_bytes(h, 1, H, G, d),
            bsa.bsa_attention_weights_workspace_bytes(h, H, G), bsa.bsa_evict_workspace_bytes(h, 1, G, 200))]
        return x

    def calls(x, stream=None):
        bsa.decode_tree(q, kt, vt, x.kc, x.vc, table, lens, par, lay, o=x.o, lse=x.lse, workspace=x.ws[0], stream=stream)
        bsa.decode_weights(q1, x.kc, x.vc, table, pos, lay, 1, x.w, o=x.o1, lse=x.lse1, workspace=x.ws[1], stream=stream)
        bsa.attention_weights(qp, kp, lsep, lay, x.wp, workspace=x.ws[2], stream=stream)
        bsa.evict(x.kc, x.vc, table, lens, x.w, lay, 200, 20, weights_out=x.wo, tokens_out=x.to, lengths_out=x.lo,
                  workspace=x.ws[3], stream=stream)

    def same(x, y):
        return all(torch.equal(getattr(x, a).view(torch.uint8), getattr(y, a).view(torch.uint8))
                   for a in ("o", "lse", "o1", "lse1", "w", "wp", "kc", "vc", "wo", "to", "lo"))

    ref, a, b = bufs(), bufs(), bufs()
    calls(ref)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s, x in ((s1, a), (s2, b)):
        calls(x, s)
    torch.cuda.synchronize()
    assert same(a, ref) and same(b, ref)
    # on a raw stream handle, allocating its own outputs and workspace there
    o, lse = bsa.decode_tree(q, kt, vt, kc, vc, table, lens, par, lay, stream=s1.cuda_stream)
    s1.synchronize()
    assert torch.equal(o, ref.o) and torch.equal(lse, ref.lse)
    # captured once, replayed on other inputs written in place
    c = bufs()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(c)
    for seed in (130, 140):
        qb = inputs.normal_bf16_bits((H, T, d), seed)
        q.copy_(to_device_bf16(qb))
        q1.copy_(q[:, 0])
        lens.fill_(850 if seed == 130 else 333)
        pos.fill_(849 if seed == 130 else 332)
        fresh = bufs()
        for name in ("o", "lse", "o1", "lse1", "w", "wp", "kc", "vc", "wo", "to", "lo"):
            getattr(c, name).copy_(getattr(fresh, name))
        torch.cuda.synchronize()
        g.replay()
        calls(fresh)
        torch.cuda.synchronize()
        assert same(c, fresh)
    bsa.bsa_get_status(lay.handle)
    del g
    lay.close()


def test_long_steps_and_cuts_refuse_replay_and_run_on_two_streams():
    """Rows too long for one kernel: a bad page and a bad length refuse their own sequence alone, calls on two
    streams and replayed ones give the bits of one call after the other."""
    n, B, batch, H, G, d, budget = 4500, 64, 2, 4, 2, 64, 1500
    lay = _layout(OL.BAND_GLOBAL, n, B, 1, dict(window=-(-n // B), global_first=0))
    kc, vc, table, th = _paged(batch, G, n, B, d, 210)
    q = to_device_bf16(inputs.normal_bf16_bits((batch * H, d), 211))
    pos = torch.tensor([n - 1, 3000], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n, 3001], dtype=torch.int32, device="cuda")
    w0 = torch.rand((batch * G, n), device="cuda")

    class Out:
        pass

    def bufs():
        x = Out()
        x.kc, x.vc, x.w = kc.clone(), vc.clone(), w0.clone()
        x.o, x.lse = torch.zeros_like(q), torch.zeros(batch * H, device="cuda")
        x.wo, x.to = torch.zeros((batch * G, n), device="cuda"), torch.zeros((batch * G, n), dtype=torch.int32, device="cuda")
        x.lo = lens.clone()
        x.ws = torch.empty(max(bsa.bsa_decode_weights_workspace_bytes(lay.handle, batch, batch * H, batch * G, d),
                               bsa.bsa_evict_workspace_bytes(lay.handle, batch, batch * G, budget)),
                           dtype=torch.uint8, device="cuda")
        return x

    def calls(x, tab=table, at=pos, ln=lens, stream=None):
        # one workspace for all: the calls of a stream follow each other
        for _ in range(2):
            bsa.decode_weights(q, x.kc, x.vc, tab, at, lay, batch, x.w, o=x.o, lse=x.lse, workspace=x.ws, stream=stream)
        bsa.evict(x.kc, x.vc, tab, ln, x.w, lay, budget, 100, weights_out=x.wo, tokens_out=x.to, lengths_out=x.lo,
                  workspace=x.ws, stream=stream)

    names = ("o", "lse", "w", "kc", "vc", "wo", "to", "lo")

    def same(x, y):
        return all(torch.equal(getattr(x, a).view(torch.uint8), getattr(y, a).view(torch.uint8)) for a in names)

    ref, a, b, c = bufs(), bufs(), bufs(), bufs()
    calls(ref)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    for s, x in ((torch.cuda.Stream(), a), (torch.cuda.Stream(), b)):
        calls(x, stream=s)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    assert same(a, ref) and same(b, ref)
    with torch.cuda.graph(g):
        calls(c)
    pos.fill_(2600)
    lens.fill_(2601)
    fresh = bufs()
    for name in names:
        getattr(c, name).copy_(getattr(fresh, name))
    torch.cuda.synchronize()
    g.replay()
    calls(fresh)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    assert same(c, fresh)
    # sequence 0 refused: by a page that does not exist, and by a position and length past the end
    past = torch.tensor([n + 1, 2601], dtype=torch.int32, device="cuda")
    bad = table.clone()
    bad[0, 7] = kc.shape[0]
    for tab, at, ln in ((bad, pos, lens), (table, past - 1, past)):
        x = bufs()
        calls(x, tab, at, ln)
        torch.cuda.synchronize()
        with pytest.raises(bsa.BsaError):
            bsa.bsa_get_status(lay.handle)
        assert torch.all(x.o[:H] == 0) and torch.all(torch.isneginf(x.lse[:H])) and torch.equal(x.w[:G], w0[:G])
        assert torch.all(x.wo[:G] == 0) and torch.all(x.to[:G] == 0) and x.lo.tolist() == [-1, budget]
        mine = table[0].long()
        assert torch.equal(x.kc[mine].view(torch.int16), kc[mine].view(torch.int16))
        for name in ("o", "lse"):
            assert torch.equal(getattr(x, name)[H:], getattr(fresh, name)[H:])
        for name in ("w", "wo", "to"):
            assert torch.equal(getattr(x, name)[G:], getattr(fresh, name)[G:])
    del g
    lay.close()


def test_wrong_tensors_are_refused():
    lay, q, kt, vt, kc, vc, table, lens, par = _small_tree(150)
    good = (q, kt, vt, kc, vc, table, lens, par)
    bsa.decode_tree(*good, lay)
    bad = {0: q.float(), 1: kt[:, :4].contiguous(), 2: vt.transpose(1, 2), 3: kc[:, :, :32].contiguous(),
           5: table.long(), 6: lens.cpu(), 7: par[:, :4].contiguous()}
    for at, x in bad.items():
        args = list(good)
        args[at] = x
        with pytest.raises((bsa.BsaError, ValueError)):
            bsa.decode_tree(*args, lay)
    w = torch.zeros((2, 1000), device="cuda")
    pos = lens - 1
    q1 = q[:, 0].contiguous()
    for x in (w.double(), w[:, :999], w[:1], w.cpu(), torch.zeros((1000, 2), device="cuda").t()):
        with pytest.raises(bsa.BsaError):
            bsa.decode_weights(q1, kc, vc, table, pos, lay, 1, x)
        with pytest.raises(bsa.BsaError):
            bsa.evict(kc, vc, table, lens, x, lay, 100, weights_out=torch.zeros_like(w), tokens_out=torch.zeros_like(w, dtype=torch.int32))
    with pytest.raises(bsa.BsaError):
        bsa.evict(kc, vc, table, lens, w, lay, 100, weights_out=w)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    lay.close()


def test_no_block_kept_at_all():
    """An explicit mask that keeps nothing: empty rows everywhere, and no weight."""
    n, B, H, G, d, T = 200, 64, 2, 1, 64, 3
    lay = bsa.Layout(OL.EXPLICIT, n, B, 1, torch.cuda.current_device(), mask=np.zeros((1, 4, 4), np.uint8))
    kc, vc, table, th = _paged(1, G, n, B, d, 160)
    q, kt, vt = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, T, d, seeds=(161, 162, 163)))
    o, lse = bsa.decode_tree(q, kt, vt, kc, vc, table, torch.tensor([150], dtype=torch.int32, device="cuda"),
                             torch.tensor([[-1, 0, 1]], dtype=torch.int32, device="cuda"), lay)
    w = torch.full((G, n), 2.0, device="cuda")
    o1, lse1 = bsa.decode_weights(q[:, 0].contiguous(), kc, vc, table,
                                  torch.tensor([150], dtype=torch.int32, device="cuda"), lay, 1, w)
    qp, kp, vp = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, n, d))
    bsa.attention_weights(qp, kp, torch.full((H, n), float("-inf"), device="cuda"), lay, w)
    torch.cuda.synchronize()
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse)) and torch.all(o1 == 0)
    assert torch.all(torch.isneginf(lse1)) and torch.all(w == 2)
    bsa.bsa_get_status(lay.handle)
    lay.close()


def test_a_serving_run():
    """Prompt, its weights, the cut, steps that add up, a drafted tree over the cut cache, and a second cut: each
    against the oracle on what the one before left."""
    n, B, H, G, d, budget, recent = 1024, 64, 4, 2, 64, 300, 40
    prompt, scale = 700, d ** -0.5
    full = dict(window=n // B, global_first=0)
    route = bsa.Layout(OL.DYADIC, prompt, B, 1, torch.cuda.current_device(), **DYADIC)
    slots = _layout(OL.BAND_GLOBAL, n, B, 1, full)
    all_blocks = OL.kept_sets(OL.BAND_GLOBAL, n, B, 1, **full)
    qb, kb, vb = inputs.qkv_bits(H, G, prompt, d, seeds=(170, 171, 172))
    q, k, v = (to_device_bf16(x) for x in (qb, kb, vb))
    o, lse = bsa.attention(q, k, v, route, scale)
    weights = torch.zeros((G, n), device="cuda")
    bsa.attention_weights(q, k, lse, route, weights, scale)
    kc, vc, table, th = _paged(1, G, n, B, d, 173)
    for c, x in ((kc, k), (vc, v)):
        pad = torch.zeros((G, 11 * B, d), dtype=torch.bfloat16, device="cuda")
        pad[:, :prompt] = x
        c[table[0, :11].long()] = pad.view(G, 11, B, d).transpose(0, 1)
    lens = torch.tensor([prompt], dtype=torch.int32, device="cuda")
    tokens = None
    for cut in range(2):
        before = _np(kc), _np(vc), weights.cpu().numpy(), None if tokens is None else tokens.cpu().numpy(), lens.tolist()
        weights, tokens, lens = bsa.evict(kc, vc, table, lens, weights, slots, budget, recent, tokens=tokens)
        torch.cuda.synchronize()
        kh, vh, wh, tkh, lh = OC.evict(before[0], before[1], th, before[4], before[2], before[3], n, budget, recent)
        np.testing.assert_array_equal(_np(kc), kh)
        np.testing.assert_array_equal(weights.cpu().numpy(), wh)
        np.testing.assert_array_equal(tokens.cpu().numpy(), tkh)
        assert lens.tolist() == lh.tolist() == [budget]
        for step in range(5):
            t = int(lens[0])
            new = to_device_bf16(inputs.normal_bf16_bits((H + 2 * G, d), 180 + 10 * cut + step))
            kc[int(th[0, t // B]), :, t % B], vc[int(th[0, t // B]), :, t % B] = new[H:H + G], new[H + G:]
            w0 = _np(weights)
            o, lse = bsa.decode_weights(new[:H].contiguous(), kc, vc, table, lens, slots, 1, weights, scale)
            torch.cuda.synchronize()
            lens = lens + 1
            kh, vh, qh = np.nan_to_num(_np(kc)), np.nan_to_num(_np(vc)), _np(new[:H])
            o_ref, lse_ref = OD.decode_step(qh, kh, vh, th, [t], all_blocks, B, scale)
            e_p = _e_p(scale, d, qh, kh, lse_ref)
            _close_o(_np(o), o_ref, e_p, vh)
            want = OC.step_weights(qh, kh, th, [t], lse_ref, all_blocks, B, scale, n)
            bound = want * (2 * e_p + 2.0 ** -20) + 2.0 ** -24 * (want + w0)
            assert np.all(np.abs(_np(weights) - w0 - want) <= bound)
        T = 6
        par = np.array([[-1, 0, 0, 1, 3, -1]], np.int32)
        tq, tk, tv = (to_device_bf16(x) for x in inputs.qkv_bits(H, G, T, d, seeds=(200 + cut, 201, 202)))
        o, lse = bsa.decode_tree(tq, tk, tv, kc, vc, table, lens, torch.from_numpy(par).cuda(), slots, scale)
        torch.cuda.synchronize()
        o_ref, lse_ref = OC.tree(_np(tq), _np(tk), _np(tv), kh, vh, th, lens.tolist(), par, all_blocks, B, scale)
        e_p = _e_p(scale, d, _np(tq), kh, lse_ref)
        _close_o(_np(o), o_ref, e_p, np.concatenate([vh.reshape(-1, d), _np(tv).reshape(-1, d)]))
        _close_lse(_np(lse), lse_ref, e_p)
        # the path 0, 1, 3 is taken: its keys and values enter the cache with no weight yet
        for x in (0, 1, 3):
            t = int(lens[0])
            kc[int(th[0, t // B]), :, t % B], vc[int(th[0, t // B]), :, t % B] = tk[:, x], tv[:, x]
            lens = lens + 1
        assert tokens[0, :budget].max() == (prompt - 1 if cut == 0 else prompt + 7)
    bsa.bsa_get_status(slots.handle)
    route.close()
    slots.close()
