"""The operators of a serving step on calls that strain what their kernels keep
beside the values (plain forms and bounds: tests/serve_ref.py, tests/layer_ref.py)."""
import numpy as np
import pytest

import weight_only_bit_block_amd as wqa
from tests import serve_ref as sref
from tests.gpu_util import note, torch_cuda
from tests.test_gpu_layer import NAN, dev, qkv, rng_for
from tests.test_gpu_serve import freqs

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norms and rotation
@pytest.mark.parametrize("d,pairs", [(64, 0), (64, 8), (64, 28), (128, 0), (128, 4), (128, 32), (128, 60)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T", [5, 1100])
def test_rope_values_that_are_not_rotated_are_kept(d, pairs, inter, T):
    """Without the norm they are copies, bit by bit, whatever stands beside them; with it each is its own product."""
    note(f"rope tail {d} {pairs} {inter} {T}")
    torch_cuda()
    rng = rng_for(110, d, pairs, T)
    host, _ = qkv(rng, T, 6, 3, d)
    x, y = host[0], host[1]
    tail = slice(2 * pairs, d)
    pos, inv = rng.integers(1, 100000, T).astype(np.int32), freqs(pairs) if pairs else np.zeros(0, np.float32)
    for a in (x, y):
        spots = rng.random(a[..., tail].shape) < 0.1
        a[..., tail][spots] = rng.choice(np.array([np.nan, np.inf, -np.inf, -0.0, 0.0, 1e-44], np.float32), int(spots.sum()))
    oq, ok = wqa.qk_norm_rope(dev(x), dev(y), dev(pos), dev(inv), norm=False, interleaved=inter, factor=1.5)
    for got, a in ((oq.cpu().numpy(), x), (ok.cpu().numpy(), y)):
        assert np.array_equal(got[..., tail].view(np.uint32), a[..., tail].view(np.uint32))
        want, lim = sref.rope(a, pos, inv, None, 0.0, False, inter, 1.5)
        assert (np.abs(got - want)[..., :2 * pairs] <= lim[..., :2 * pairs]).all()
    # with the norm: a weight that is not finite belongs to its own value
    host, (q, _, _) = qkv(rng, T, 6, 3, d)
    for bad in (NAN, np.inf):
        w = rng.standard_normal(d).astype(np.float32)
        w[[2 * pairs, d - 1]] = bad
        got = wqa.qk_norm_rope(q, None, dev(pos), dev(inv), q_weight=dev(w), interleaved=inter)[0].cpu().numpy()
        own = np.zeros(d, bool)
        own[[2 * pairs, d - 1]] = True
        assert not np.isfinite(got[..., own]).any()
        want, lim = sref.rope(host[0], pos, inv, np.where(own, 1, w).astype(np.float32), 1e-6, True, inter, 1.0)
        assert (np.abs(got - want)[..., ~own] <= lim[..., ~own]).all()
