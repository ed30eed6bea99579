"""The cosines and sines of the rotation, seen as the rotated pair (1, 0), against float64.

Tolerance, derived: the phase is exact to 2^-32 of a turn (cut off); the rest of a quarter turn is at most 1/4 half turn,
so it is off by 2^-27 half turns in fp32; the half-turn functions are off by one unit of the result, at most 2^-23 of
it.  In radians pi (2^-31 + 2^-27) + 2^-23 |value|."""
import numpy as np
import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("H", [1, 2])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_cosine_and_sine(dev, layout, H, inverse):
    d, T = 64, 20000
    rng = np.random.default_rng(H)
    pos = np.concatenate([np.arange(4000), rng.integers(-2 ** 31, 2 ** 31, T - 4000)]).astype(np.int32)
    plan = dsa.Rope.make(d, layout=layout)
    x = torch.zeros((T, H, d), device=dev)
    first = (slice(0, d, 2), slice(1, d, 2)) if layout == "interleaved" else (slice(0, d // 2), slice(d // 2, d))
    x[..., first[0]] = 1.0
    out = dsa.rope(plan, torch.from_numpy(pos).to(dev), x, torch.empty_like(x), inverse=inverse).double().cpu().numpy()
    turns = plan.turns.cpu().numpy().view(np.uint64)
    phase = pos.astype(np.int64).view(np.uint64)[:, None] * turns[None, :]         # modulo one turn
    angle = (phase.view(np.int64).astype(np.float64) * 2.0 ** -64 * 2 * np.pi)[:, None, :]
    for part, want in ((first[0], np.cos(angle)), (first[1], np.sin(-angle if inverse else angle))):
        err = np.abs(out[..., part] - want)
        tol = np.pi * (2.0 ** -31 + 2.0 ** -27) + 2.0 ** -23 * np.abs(want)
        assert np.all(err <= tol), float((err / tol).max())
