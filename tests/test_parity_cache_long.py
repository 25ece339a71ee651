"""Cache attention for many rows whose thread blocks go through many key blocks
each, and the d = 64 forms of the tests for tokens that are not finite, of
repeated calls and of waits that run out.

The reference is the definition in 64 bits on the GPU; the bars are those that
test_parity_cache.py derives.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C
from test_parity_cache import DEV, Fwd, _bytes_of, _status_ok, _v, ints

pytestmark = pytest.mark.gpu


class Long:
    """Streams whose tables list the same few pages again and again."""

    def __init__(self, d, kv_heads, group, pt, steps, frame=0, seed=0, pool_tokens=8192):
        self.V = _v()
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        pages = pool_tokens // pt
        self.d, self.pt, self.steps, self.frame, self.group = d, pt, steps, frame, group
        x = torch.randn((2, pages, kv_heads, pt, d), generator=gen, device=DEV) * 100
        self.kc, self.vc = x.clamp(-448, 448).to(torch.float8_e4m3fn)
        self.ks, self.vs = torch.exp2(torch.randint(-9, -4, (2, pages, kv_heads, pt // 16), generator=gen, device=DEV).float())
        width = -(-max(length for length, _ in steps) // pt)
        self.table = torch.randint(0, pages, (len(steps), width), generator=gen, device=DEV).to(torch.int32)
        self.starts = np.cumsum([0] + [n for _, n in steps])
        self.rows, self.max_new = int(self.starts[-1]), max(n for _, n in steps)
        self.q = torch.randn((self.rows, kv_heads * group, d), generator=gen, device=DEV).to(torch.bfloat16)
        self.geom = self.V.make_cache_geom(len(steps), kv_heads * group, kv_heads, d, pages, pt, width, frame)
        self.args = ints(self.starts), ints([x for x, _ in steps]), self.table, self.kc, self.vc, self.ks, self.vs
        self.scale = 1 / math.sqrt(d)

    def run(self):
        o = torch.full_like(self.q, 7.5)
        lse = torch.full(o.shape[:2], 7.5, device=DEV)
        ws = torch.full((self.V.vattn_cache_workspace_size(self.geom, self.rows, self.max_new),), 0xff, dtype=torch.uint8,
                        device=DEV)
        self.V.vattn_cache_fwd(self.geom, self.q, *self.args, self.scale, self.max_new, o, lse, ws)
        _status_ok(self.V)
        return o, lse

    def check(self, o, lse):
        for s, (length, n) in enumerate(self.steps):
            if n == 0:
                continue
            pages = self.table[s, :-(-length // self.pt)].long()
            a0, a1 = int(self.starts[s]), int(self.starts[s + 1])
            pos = torch.arange(length, device=DEV)
            seen = torch.ones((n, length), dtype=torch.bool, device=DEV)
            if self.frame:
                at = length - n + torch.arange(n, device=DEV)
                seen = pos // self.frame <= at[:, None] // self.frame
            for h in range(self.kc.shape[1]):
                k, v = (c[pages, h].double().flatten(0, 1)[:length] *
                        f[pages, h].double().repeat_interleave(16, 1).flatten()[:length, None]
                        for c, f in ((self.kc, self.ks), (self.vc, self.vs)))
                for g in range(self.group):
                    q = self.q[a0:a1, h * self.group + g].double()
                    x = (q @ k.T * self.scale).masked_fill(~seen, -math.inf)
                    z = torch.logsumexp(x, -1)
                    p = torch.exp(x - z[:, None])
                    ref, a = p @ v, p @ v.abs()
                    delta = 2.0 ** -16 * self.scale * q.abs().amax(-1) * k.abs().sum(-1).max()
                    bar = 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2 * delta[:, None]) * a + 2.0 ** -20 * v.abs().max()
                    got, gl = o[a0:a1, h * self.group + g].double(), lse[a0:a1, h * self.group + g].double()
                    assert bool(((got - ref).abs() <= bar).all()), (s, h, g)
                    assert bool(((gl - z).abs() <= delta + 2.0 ** -18 * (1 + z.abs())).all()), (s, h, g)


LONG = [
    # one tile of rows a thread block, alternate key blocks to the two groups
    (16, 2, 64, [(8200 + 131 * i, 17 + i) for i in range(40)], 1),
    # two tiles of rows, and a second one that is partly or wholly empty
    (16, 1, 16, [(9000 + 77 * i, 130 - 20 * (i % 6)) for i in range(40)], 0),
    (8, 2, 128, [(12000 + 500 * i, 520 - 60 * (i % 8)) for i in range(16)], 1),
    (4, 1, 32, [(30000, 900), (17, 5), (24000, 300), (9000, 129)] * 12, 40),
]


@pytest.mark.parametrize("case", LONG, ids=range(len(LONG)))
@pytest.mark.parametrize("d", [64, 128])
def test_many_key_blocks_a_thread_block(d, case):
    """More items than are split: each thread block goes through 64 to 235 key blocks."""
    kv_heads, group, pt, steps, frame = case
    f = Long(d, kv_heads, group, pt, steps, frame, seed=d + pt)
    o, lse = f.run()
    f.check(o, lse)
    for _ in range(3):
        o2, lse2 = f.run()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128])
def test_one_stream_over_many_keys(d):
    """One stream, its keys split; and one whose split items follow unsplit ones."""
    for kv_heads, steps in ((2, [(40000, 150)]), (24, [(9000, 3000)])):
        f = Long(d, kv_heads, 1, 64, steps, 1, seed=kv_heads)
        f.check(*f.run())


@pytest.mark.parametrize("n", [20, 140])
def test_a_token_that_is_not_finite_spoils_only_who_sees_it_d64(n):
    f = Fwd(d=64, kv_heads=2, group=1, pt=32, steps=[(700, n), (200, n)], frame=1, seed=5)
    page, row = int(f.table[0, 650 // 32]), 650 % 32
    _bytes_of(f.kc)[page, 1, row] = 0x7f
    _bytes_of(f.vc)[page, 1, row] = 0
    f.q[f.starts[1], 0, 3] = math.nan
    o, lse = f.run()
    bad = torch.zeros((f.rows, 2), dtype=torch.bool, device=DEV)
    bad[:n, 1] = torch.from_numpy(C.seen(1, 0, 700, n)[:, 650]).to(DEV)
    bad[f.starts[1], 0] = True
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    assert torch.equal(torch.isnan(lse), bad)
    _bytes_of(f.kc)[page, 1, row] = 0
    f.q[f.starts[1], 0, 3] = 0
    f.check(*f.run())


@pytest.mark.parametrize("n", [60, 200])
def test_bounded_waits_run_out_d64(n):
    """The load warp's first arrival withheld: the kernel gives up, reports it and leaves the device usable."""
    V = _v()
    f = Fwd(d=64, kv_heads=1, group=1, pt=64, steps=[(400, n)], seed=15)
    want = f.run()
    o, lse, ws = f.outputs()
    V.vattn_debug_set(V.binding.VATTN_DEBUG_SKIP_ARRIVAL, 20_000_000)
    try:
        f.call(o, lse, ws)
        assert V.vattn_get_status() == V.binding.VATTN_ERR_DEVICE_TIMEOUT
    finally:
        V.vattn_debug_set(0, 0)
    assert (o[f.n:] == 7.5).all()
    got = f.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
