"""Masks whose query blocks often keep nothing, with many more work items than
the GPU runs at once: the kernels take up one item without kept blocks after
the other, and items with some between them.  Against the fp64 oracle;
gradients with the tolerances of their other parity tests.

Rows of one or a few keys have outputs as large as a value, so o's bound goes
by its size: P enters the product rounded to bf16, by at most 2^-8 of itself
(the sum l is taken of P before that), P itself is off by e_p (as derived in
test_gpu_cache.py, for P and again for l), and o is rounded once:
  |o - o_ref| <= half a bf16 step of o + (2^-8 + 2 e_p) sum_u p_u |v_u|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_sparse_long_bsa_b200 as bsa
from block_sparse_long_bsa_b200 import inputs
from oracle import attention as OA
from oracle import backward as BW
from oracle import layouts as OL

from gpu_common import bf16_half_ulp, default_scale, device_inputs, to_device_bf16
from test_gpu_backward import assert_grad_close
from test_gpu_cache import _close_lse, _e_p, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bsa.load_library()


CASES = [
    # n, B, layout heads, heads, kv heads, d, share of rows that keep nothing, share of blocks the others keep
    (2117, 64, 1, 18, 2, 64, 0.2, 0.87),
    (1607, 128, 34, 34, 2, 128, 0.2, 0.74),
    (2233, 64, 1, 27, 3, 128, 0.3, 0.15),
    (2048, 64, 1, 32, 4, 128, 0.9, 0.5),          # two heads an item
    (2048, 128, 64, 64, 4, 64, 0.95, 0.5),
    (1500, 64, 40, 40, 8, 64, 0.98, 0.3),         # most layout heads keep nothing at all
    (1100, 64, 1, 64, 8, 128, 1.0, 0.5),          # no row keeps anything
    (2000, 64, 20, 20, 4, 64, 0.6, 0.05),         # items of one or two blocks
]


def _mask(n, B, L, empty, keep, seed):
    nb = -(-n // B)
    rng = np.random.default_rng(seed)
    m = np.tril(rng.random((L, nb, nb)) < keep)
    m |= np.eye(nb, dtype=bool)[None] & (rng.random((L, nb, 1)) < 0.5)
    m[rng.random((L, nb)) < empty] = False
    sets = [[set(np.nonzero(m[h, i])[0].tolist()) for i in range(nb)] for h in range(L)]
    return m.astype(np.uint8), sets


def _layout(case):
    n, B, L, H, G, d, empty, keep = case
    mask, sets = _mask(n, B, L, empty, keep, n)
    return bsa.Layout(OL.EXPLICIT, n, B, L, torch.cuda.current_device(), mask=mask), sets


@pytest.mark.parametrize("case", CASES)
def test_forward_with_empty_rows(case):
    n, B, L, H, G, d, empty, keep = case
    lay, sets = _layout(case)
    (qb, kb, vb), (q, k, v) = device_inputs(H, G, n, d, seeds=(500, 501, 502))
    scale, runs = default_scale(d), []
    for _ in range(6):                              # the order in which items are taken differs from run to run
        runs.append(bsa.attention(q, k, v, lay))
        torch.cuda.synchronize()
        bsa.bsa_get_status(lay.handle)
    o, lse = runs[0]
    assert all(torch.equal(x, o) and torch.equal(y, lse) for x, y in runs)
    qh, kh, vh = (inputs.bf16_bits_to_f64(x) for x in (qb, kb, vb))
    o_ref, lse_ref = OA.forward_dense(qh, kh, vh, sets, B, scale)
    e_p = _e_p(scale, d, qh, kh, lse_ref)
    _close_lse(_np(lse), lse_ref, e_p)
    bound = bf16_half_ulp(_np(o)) + (2.0 ** -8 + 2 * e_p) * OA.forward_dense(qh, kh, np.abs(vh), sets, B, scale)[0]
    assert np.all(np.abs(_np(o) - o_ref) <= bound), (np.abs(_np(o) - o_ref) / bound).max()
    assert np.all(_np(o)[~np.isfinite(lse_ref)] == 0)
    lay.close()


@pytest.mark.parametrize("case", CASES[:6])
def test_prompt_weights_with_empty_rows(case):
    """The sums of each key/value head are the number of its query rows that read anything."""
    n, B, L, H, G, d, empty, keep = case
    lay, _ = _layout(case)
    _, (q, k, v) = device_inputs(H, G, n, d, seeds=(510, 511, 512))
    _, lse = bsa.attention(q, k, v, lay)
    w, w2 = bsa.attention_weights(q, k, lse, lay), bsa.attention_weights(q, k, lse, lay)
    torch.cuda.synchronize()
    bsa.bsa_get_status(lay.handle)
    rows = torch.isfinite(lse).view(G, -1).sum(1).double()
    # a probability is off by 2e-5 of itself here at most (norms up to 12), a row's sum by no more
    assert torch.equal(w, w2) and torch.all((w.double().sum(1) - rows).abs() <= 3e-5 * rows)
    lay.close()


@pytest.mark.parametrize("case", CASES)
def test_gradients_with_empty_rows(case):
    n, B, L, H, G, d, empty, keep = case
    lay, sets = _layout(case)
    (qb, kb, vb), (q, k, v) = device_inputs(H, G, n, d, seeds=(500, 501, 502))
    dob = inputs.normal_bf16_bits((H, n, d), 503)
    do, scale, runs = to_device_bf16(dob), default_scale(d), []
    o, lse = bsa.attention(q, k, v, lay)
    for _ in range(6):
        runs.append(bsa.attention_backward(q, k, v, o, lse, do, lay))
        torch.cuda.synchronize()
        bsa.bsa_get_status(lay.handle)
    assert all(torch.equal(r[0], runs[0][0]) for r in runs) and torch.all(runs[0][0][torch.isneginf(lse)] == 0)
    ref = BW.backward_dense(*(inputs.bf16_bits_to_f64(x) for x in (qb, kb, vb, dob)), sets, B, scale)
    for r in runs:
        for name, g, want in zip(("dq", "dk", "dv"), r, ref):
            assert_grad_close(g.cpu().numpy(), want, f"{case} {name}")
    lay.close()
