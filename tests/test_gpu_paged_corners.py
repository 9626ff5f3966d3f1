"""GPU parity of the paged operators where they can go wrong: blocks without
a key tile, score factors at the ends of fp32, variants chosen by the table's
size, and bytes that no other test looks at."""

import numpy as np
import pytest

from test_gpu_paged_attention import Problem, rt  # noqa: F401  (rt: the fixture)

pytestmark = pytest.mark.gpu


def repeat(p, times):
    """The same bits from call to call."""
    out, lse = p.out.clone(), p.lse.clone()
    torch = p.rt[2]
    for _ in range(times):
        p.out.fill_(5.0)
        p.lse.fill_(5.0)
        p.run()
        assert torch.equal(out, p.out) and torch.equal(lse, p.lse)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,lens,causal", [
    # keys in no split of any block, with the keys split (few units) ...
    (8, 2, [(300, 0), (257, 3), (1, 5)], True), (8, 2, [(300, 0), (300, 0)], False),
    # ... and with the units filling the SMs
    (32, 8, [(300, 0), (300, 2), (64, 900)], True), (32, 8, [(300, 0), (300, 0), (40, 7)], False),
    # more splits than a short sequence has key tiles
    (8, 2, [(64, 1500), (64, 100), (64, 130), (33, 1)], False),
    (8, 2, [(64, 1500), (64, 100), (64, 130), (64, 9)], True)])
def test_blocks_without_a_key_tile(rt, hd, hq, hkv, lens, causal):  # noqa: F811
    """Hundreds of live rows in a block that has no key to read."""
    p = Problem(rt, np.random.default_rng(31), lens, hq, hkv, hd, 32, causal)
    p.run()
    p.check()
    repeat(p, 10)


@pytest.mark.parametrize("Lq", [1, 3, 60])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("gain,scale", [(2.0 ** -80, 0.0), (2.0 ** -126, 0.0), (2.0 ** 100, 0.0), (2.0 ** 120, 0.0),
                                        (2.0 ** -100, 1e-30), (2.0 ** -110, -1e-37), (1.0, 1e-45)])
def test_factors_below_fp32(rt, Lq, hd, gain, scale):  # noqa: F811
    """Scale times |q| from nothing to below the least fp32 number, under a
    mask: every visible key weighs the same."""
    p = Problem(rt, np.random.default_rng(32), [(Lq, 150), (1, 70), (Lq, 1)], 4, 2, hd, 16, scale=scale, q_gain=gain)
    p.run()
    p.check()
