"""Query rows that are not finite and see no key: empty like any other row that
sees none (O = 0, LSE = -inf), whatever the other rows of their tile see."""
import math

import pytest
import torch

from oracle import cache_oracle as C
from test_parity_cache import DEV, Fwd, _status_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv_heads,group", [(2, 1), (1, 2)])
@pytest.mark.parametrize("steps,frame,window", [
    ([(2, 5)], 1, 0),                        # few rows, the first three see nothing
    ([(0, 4), (9, 3)], 1, 0),                # a stream without keys
    ([(30, 70)], 16, 0),                     # one tile, mixed
    ([(600, 900)], 1, 0),                    # whole tiles that see nothing, one mixed, others not
    ([(0, 140), (300, 20)], 1, 0),
    ([(90, 100), (2000, 90), (50, 260)] * 4, 7, 3),
    ([(1500, 1590)], 1, 0),                  # one stream: split keys
])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing_are_empty_whatever_their_query(d, steps, frame, window, kv_heads, group):
    f = Fwd(d=d, kv_heads=kv_heads, group=group, pt=32, steps=steps, frame=frame, window=window, seed=d)
    bad = torch.zeros(f.rows, dtype=torch.bool, device=DEV)
    bad[:f.n:3] = True
    clean = f.q.clone()
    o, lse = f.run()
    f.q[bad, :, 5] = math.nan
    f.q[bad, 0, 7] = math.inf
    o2, lse2 = f.run()
    _status_ok(f.V)
    empty = torch.cat([torch.from_numpy(~C.seen(frame, window, length, n).any(1)) for length, n in steps if n]).to(DEV)
    assert (bad[:f.n] & empty).any()
    nan = bad.clone()
    nan[:f.n] &= ~empty
    assert torch.isnan(o2[nan]).all() and torch.isnan(lse2[nan]).all()
    assert torch.equal(o2[~nan], o[~nan]) and torch.equal(lse2[~nan], lse[~nan])
    assert (o2[:f.n][empty] == 0).all() and (lse2[:f.n][empty] == -math.inf).all()
    f.q.copy_(clean)
    f.check(o, lse)
