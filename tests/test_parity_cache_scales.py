"""V's scales as far apart as the header allows, 2^100: the weights of the
blocks with small scales count in full.

A weight is 2^(x - m + 7) with x = score + log2(scale) and m at most the largest
x; it leaves fp32 below 2^-126, so at 2^100 a token counts down to 2^-33 of the
largest weight.  Beside the bars of test_parity_cache.py, which hold: x is off
by half a step of numbers below 128, 2^-18, or 2^-18.5 of a weight.
"""
import math

import numpy as np
import pytest
import torch

from test_parity_cache import DEV, Fwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("steps,frame", [([(700, 1), (90, 1)], 0), ([(5000, 1)], 0), ([(400, 6)], 1), ([(300, 60)], 1),
                                         ([(900, 200)], 0), ([(9000, 40)], 1), ([(700, 300), (40, 9)] * 3, 1)],
                         ids=["one", "one split", "few", "many, one tile", "many", "many split", "streams"])
def test_scales_of_v_far_apart(d, steps, frame):
    f = Fwd(d=d, kv_heads=2, group=1, pt=32, steps=steps, frame=frame, seed=21)
    gen = torch.Generator(device=DEV).manual_seed(d)
    for exponents in ((-40, 60), (19, 119), (-40, 60, -10, 25)):
        pick = torch.randint(0, len(exponents), f.vs.shape, generator=gen, device=DEV)
        scale = torch.exp2(torch.tensor(exponents, dtype=torch.float64, device=DEV)[pick]).float()
        f.vs = torch.where(torch.isnan(f.vs), f.vs, scale)
        if exponents[1] == 119:        # stay within what bf16 holds
            f.vc = (f.vc.float() * 2.0 ** -8).to(torch.float8_e4m3fn)
        f.check(*f.run())


@pytest.mark.parametrize("n", [1, 40, 200])
def test_a_block_of_zeros_next_to_huge_values(n):
    """Half of the tokens are zeros as vattn_cache_append stores them, the others 2^68: O halves, LSE does not."""
    f = Fwd(d=128, kv_heads=1, group=1, pt=16, steps=[(320, n)], seed=3)
    f.kc.view(torch.uint8)[f.table[0, :20]] = 0                  # every score is 0
    f.vc = torch.full(f.vc.shape, 256.0, device=DEV).to(torch.float8_e4m3fn)
    for i, page in enumerate(f.table[0, :20]):
        f.vs[page] = 2.0 ** -40 if i % 2 else 2.0 ** 60
        if i % 2:
            f.vc.view(torch.uint8)[page] = 0
    o, lse = f.run()
    assert (o[:n].double() == 2.0 ** 67).all()
    np.testing.assert_allclose(lse[:n].double().cpu().numpy(), math.log(320), rtol=0, atol=2.0 ** -18 * 7)
