"""norm_plain (64 bits on the inputs' device, gradients by automatic differentiation) against the
oracle, on the host."""
import numpy as np
import pytest
import torch

import norm_plain as plain
from oracle import nabla_oracle as O


@pytest.mark.parametrize("norm,branch", [("layer", ""), ("rms", "u"), ("layer", "rms"),
                                         ("rms", "layer")])
@pytest.mark.parametrize("weights", [True, False])
def test_against_the_oracle(norm, branch, weights):
    c = plain.Inputs(2, 12, 24, torch.float32, norm, branch, 3, weights=weights, seed=1,
                     device="cpu")

    def host(t):
        return None if t is None else t.double().numpy()

    mods = [host(t) for t in (c.gate, c.scale, c.shift, c.w, c.pw)]
    rest = (c.norm, c.post, c.rs, plain.EPS)
    s, y = O.block_norm(host(c.x), host(c.u), *mods, *rest)
    got = plain.forward(c)
    assert ("s" in got) == (c.u is not None)
    if "s" in got:
        np.testing.assert_allclose(got["s"][0], s, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(got["y"][0], y, rtol=1e-12, atol=1e-13)
    want = O.block_norm_bwd(s, host(c.u), host(c.dsum), host(c.dy), *mods, *rest)
    got = plain.backward(c, torch.from_numpy(np.asarray(s)))
    for name, ref in zip(plain.GRADS, want):
        assert (name in got) == (ref is not None), name
        if ref is not None:
            value, size = got[name]
            np.testing.assert_allclose(value, ref, rtol=1e-11, atol=1e-12, err_msg=name)
            assert size.shape == value.shape and bool((size >= 0.999 * value.abs()).all()), name
