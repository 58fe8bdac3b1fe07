"""decode, gather_kv and merge_states on the GPU: precision of the probabilities, calls on a stream
with memory of their own, mixed batches, and forms in combination (references and bounds that are
not derived here: serving_helpers.py)."""
import numpy as np
import pytest
import torch

import serving_helpers as S
from gpu_helpers import ensure_built
from test_gpu_serving import _compare, _decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


# ---------------------------------------------------------------------------------- precision

def _unit_keys(cache):
    """Every K code +-1 and every K descale 2^-3, in the pages and in the lists."""
    one = lambda c: np.where((c & 0x7f) == 0x7f, c, (c & 0x80) | 0x38).astype(np.uint8)
    cache.k_pages = one(cache.k_pages)
    cache.k = [one(c) for c in cache.k]
    cache.kd_pages = np.where(np.isnan(cache.kd_pages), cache.kd_pages, 0.125).astype(np.float32)
    cache.kd = [np.full_like(d, 0.125) for d in cache.kd]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lens,N1,N2,form", [
    ([2, 3, 5, 8, 12], 8, 1, None), ([2, 7, 33], 32, 2, None), ([4, 9, 200], 16, 1, "mask"),
    ([3, 6, 140], 8, 1, "index")])
def test_decode_probabilities_keep_their_bits(lens, N1, N2, form, q8):
    """Scores that fp32 holds exactly up to one product: queries and K codes are +-1, so q . k is an
    integer below 2^7, and K's descale is 2^-3.  What is left of a weight's error: the rounding of
    scale * log2(e) and of its product with the integer (|s| log2(e) < 24: 2^-20 each), of the
    reference and of the difference (2^-20 each), 2^-22 of the exponential: together below 2^-18 of
    the weight, 2^-17 of the quotient.  Sums over n tokens add at most n 2^-21 (one fp32 rounding
    and a truncated alignment a term, twice).  With A = sum_j p_j |v_j| / l the result is off by
    2^-8 |O| + (2^-16 + n 2^-21) A, where few tokens of mixed signs make |O| far smaller than A; one
    rounding of the weights to 11 bits is 2^-12 A and stands out."""
    cache = S.Cache(sum(lens) + N1, lens, N2, 32)
    _unit_keys(cache)
    rng = np.random.default_rng(N1)
    sign = rng.choice([-1.0, 1.0], (len(lens), N1, 128))
    if q8:
        q = torch.from_numpy(np.where(sign < 0, 0xb8, 0x38).astype(np.uint8))
        qd = torch.ones(len(lens), N1)
    else:
        q, qd = torch.from_numpy(sign).to(torch.bfloat16), None
    on = None
    if form:
        on = rng.random((len(lens), N1, -(-max(lens) // 128))) < 0.5
        on[:, ::2, 0] = True
    out, lse = _decode(cache, q, qd, on, form or "mask", scale=1.0)
    for b, n in enumerate(lens):
        k, v = cache.rows(b)
        for h in range(N1):
            take = np.ones(n, bool) if on is None else np.repeat(on[b, h], S.TILE)[:n]
            if not take.any():
                assert (out[b, h] == 0).all() and lse[h, b] == S.NEG_FLT_MAX
                continue
            kk, vv = k[h // (N1 // N2)][take], v[h // (N1 // N2)][take]
            s = kk @ sign[b, h]
            p = np.exp(s - s.max())
            O, A = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
            bound = 2.0 ** -8 * np.abs(O) + (2.0 ** -16 + n * 2.0 ** -21) * A
            S.within(out[b, h], O, bound, f"O of {b}, {h}")
            z = s.max() + np.log(p.sum())
            assert abs(float(lse[h, b]) - z) <= 2.0 ** -16 + n * 2.0 ** -21 + 2.0 ** -22 * abs(z)
