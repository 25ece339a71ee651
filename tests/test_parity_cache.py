"""The 8-bit key/value cache on the GPU against the fp64 oracle.

Bars.  Plans and cache bytes are equal, bit for bit: every step of them is
exact or one rounding that both sides define alike.  Attention: the keys and
values are exact (byte times a power of two), so what remains is
  - the query's representation and the fp32 sums: a score is off by at most
    delta = 2^-16 * scale * max|q| * max_j sum_c |k_jc|;
  - P rounded to 11 bits before P V: 2^-11 of a = sum_j p_j |v_j|, twice that
    with the other roundings of a weight;
  - weights below 2^-24 of the largest, which may be dropped: 2^-20 max|v|;
  - O rounded to bf16: half a step, 2^-8 |O|.
So |O - ref| <= 2^-8 |ref| + (2^-10 + 2 delta) a + 2^-20 max|v| and
|LSE - ref| <= delta + 2^-18 (1 + |ref|).
"""
import math
import random

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _v():
    import video_dit_local_b200 as V
    return V


def _status_ok(V):
    assert V.vattn_get_status() == 0, V.vattn_last_error()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------

class Planner:
    """State on the device, and the same state in the oracle."""

    def __init__(self, streams, pt, width, pages, max_tokens, seed=0, in_place=True):
        self.V = _v()
        self.geom = self.V.make_cache_geom(streams, 1, 1, 128, pages, pt, width)
        self.args = (pt, width, pages)
        self.max_tokens = max_tokens
        order = np.random.default_rng(seed).permutation(pages)
        self.host = dict(lens=[0] * streams, table=np.full((streams, width), -1), free=order.copy(), n_free=pages)
        self.lens, self.table, self.free, self.n_free = (ints(self.host["lens"]), ints(self.host["table"]),
                                                         ints(order), ints([pages]))
        self.lens_out = self.lens if in_place else torch.full_like(self.lens, -7)
        self.n_free_out = self.n_free if in_place else torch.full_like(self.n_free, -7)
        self.starts = torch.full((streams + 1,), -7, dtype=torch.int32, device=DEV)
        self.slots = torch.full((max_tokens,), -7, dtype=torch.int32, device=DEV)
        self.result = torch.full((4,), -7, dtype=torch.int32, device=DEV)

    def step(self, new, check=True):
        V, h = self.V, self.host
        V.vattn_cache_plan(self.geom, ints(new), self.lens, self.table, self.free, self.n_free, self.lens_out,
                           self.n_free_out, self.starts, self.slots, self.result)
        st, lens, table, free, n_free, starts, slots, result = C.plan(*self.args, new, h["lens"], h["table"], h["free"],
                                                                      h["n_free"], self.max_tokens)
        if check:
            assert self.result.tolist() == result
            assert self.lens_out.tolist() == lens and self.n_free_out.tolist() == [n_free]
            assert self.starts.tolist() == starts
            assert self.slots.tolist() == slots
            assert np.array_equal(self.table.cpu().numpy(), table)
            top = max(n_free, 0)            # entries above the top are scratch
            assert np.array_equal(self.free.cpu().numpy()[:top], free[:top])
        self.host = dict(lens=lens, table=table, free=free, n_free=n_free)
        if self.lens_out is not self.lens:
            self.lens.copy_(self.lens_out)
            self.n_free.copy_(self.n_free_out)
        return st


@pytest.mark.parametrize("streams,pt,width,pages,top,in_place", [
    (1, 16, 3, 3, 20, True), (5, 16, 8, 24, 40, False), (33, 32, 6, 150, 70, True), (1025, 64, 5, 3000, 90, True),
    (2100, 16, 4, 5000, 9, False), (3, 128, 300, 700, 9000, True)])
def test_plan_steps_equal_the_oracle(streams, pt, width, pages, top, in_place):
    rng = random.Random(streams)
    p = Planner(streams, pt, width, pages, streams * top, in_place=in_place)
    got = set()
    for i in range(12):
        st = p.step([rng.choice([-1, 0, 1, 1, rng.randrange(top), top]) for _ in range(streams)])
        got.add(st)
        if st:                                     # make room
            assert p.step([-1 if rng.random() < 0.7 else 0 for _ in range(streams)]) == 0
    assert 0 in got
    _status_ok(p.V)


def test_plan_verdicts_leave_the_state_alone():
    V = _v()
    p = Planner(4, 16, 4, 9, 70)
    assert p.step([16, 17, 1, 0]) == 0
    assert p.step([0, 0, 0, 64]) == 0                       # the stream's table row is full now
    assert p.step([0, 0, 0, 1]) == V.VATTN_PLAN_TABLE_FULL
    assert p.step([16, 0, 16, 0]) == V.VATTN_PLAN_NO_PAGES
    assert p.step([40, 31, 0, -1]) == V.VATTN_PLAN_NO_SLOTS
    assert p.step([16, 0, 16, -1]) == 0                     # pages of a stream that ends serve the same step
    p.lens[1] = 65
    p.host["lens"][1] = 65
    assert p.step([0, 0, 0, 0]) == V.VATTN_PLAN_BAD_STATE
    p.lens[1] = 17
    p.host["lens"][1] = 17
    p.table[1, 1] = 9
    p.host["table"][1, 1] = 9
    assert p.step([0, -1, 0, 0]) == V.VATTN_PLAN_BAD_STATE
    p.table[1, 1] = -1
    p.host["table"][1, 1] = -1
    assert p.step([0, -1, 0, 0]) == V.VATTN_PLAN_BAD_STATE
    p.n_free[0] = -1
    p.host["n_free"] = -1
    assert p.step([0, 0, 0, 0]) == V.VATTN_PLAN_BAD_STATE
    _status_ok(V)


def test_plan_without_slots():
    p = Planner(2, 16, 4, 9, 0)
    assert p.step([0, 0]) == 0
    assert p.step([1, 0]) == p.V.VATTN_PLAN_NO_SLOTS


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def _bytes_of(c):
    return c.view(torch.uint8)


def _values(c):
    return c.float().double().cpu().numpy()


def _pool(rng, pages, heads, pt, d, lo=-9, hi=-5):
    """A pool of finite random e4m3 bytes with random scales."""
    x = torch.from_numpy(rng.normal(size=(pages, heads, pt, d)) * 100).clamp(-448, 448).float()
    c = x.to(torch.float8_e4m3fn).to(DEV)
    s = torch.from_numpy(2.0 ** rng.integers(lo, hi + 1, size=(pages, heads, pt // 16))).float().to(DEV)
    return c, s


def _bf16(rng, shape, std=1.0):
    return torch.from_numpy(rng.normal(size=shape) * std).to(torch.bfloat16)


def _chunks_slots(rng, pt, pages, chunks):
    """Slots of streams that hold `held` tokens and get `n` more, pages in random order."""
    order = list(rng.permutation(pages))
    slots = []
    for held, n in chunks:
        mine = [order.pop() for _ in range(-(-(held + n) // pt))]
        slots += [int(mine[p // pt]) * pt + p % pt for p in range(held, held + n)]
    return slots


def _append_case(d, heads, pt, chunks, seed, tweak=None, fused=True, drop=()):
    V = _v()
    rng = np.random.default_rng(seed)
    pages = sum(-(-(a + b) // pt) for a, b in chunks) + 3
    slots = _chunks_slots(rng, pt, pages, chunks)
    for i in drop:
        slots[i] = -1
    n = len(slots)
    qkv = _bf16(rng, (n, 4 * heads, d))
    qkv *= torch.exp2(torch.from_numpy(rng.integers(-4, 5, size=(n, 4 * heads, 1))).float()).to(torch.bfloat16)
    if tweak:
        tweak(qkv, heads)
    dev = qkv.to(DEV)
    k, v = dev[:, 2 * heads:3 * heads], dev[:, 3 * heads:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    kc, ks = _pool(rng, pages, heads, pt, d)
    vc, vs = _pool(rng, pages, heads, pt, d)
    want = C.append(qkv[:, 2 * heads:3 * heads].double().numpy(), qkv[:, 3 * heads:].double().numpy(), slots,
                    _values(kc), _values(vc), ks.double().cpu().numpy(), vs.double().cpu().numpy())
    g = V.make_cache_geom(1, heads, heads, d, pages, pt, 1)
    V.vattn_cache_append(g, k, v, ints(slots), kc, vc, ks, vs)
    _status_ok(V)
    for got, w in zip((_values(kc), _values(vc), ks.double().cpu().numpy(), vs.double().cpu().numpy()), want):
        np.testing.assert_array_equal(got, w)
    # once more on the same state: the same bytes again
    was = [_bytes_of(kc).clone(), _bytes_of(vc).clone()]
    V.vattn_cache_append(g, k, v, ints(slots), kc, vc, ks, vs)
    assert torch.equal(was[0], _bytes_of(kc)) and torch.equal(was[1], _bytes_of(vc))


CHUNKS = [
    [(0, 1)], [(15, 1)], [(16, 1)], [(7, 30)], [(0, 16), (0, 17), (0, 15)], [(3, 200), (129, 1), (64, 64), (1, 1)],
    [(i, 1) for i in range(40)], [(i % 17, 1 + i % 5) for i in range(60)],
]


@pytest.mark.parametrize("chunks", CHUNKS, ids=range(len(CHUNKS)))
@pytest.mark.parametrize("d,heads,pt", [(128, 3, 16), (64, 2, 64), (128, 1, 128), (64, 5, 32)])
def test_append_equals_the_oracle(d, heads, pt, chunks):
    _append_case(d, heads, pt, chunks, seed=d + pt)


def test_append_dense_tensors_and_skipped_tokens():
    _append_case(128, 2, 32, [(3, 40), (0, 20)], seed=1, fused=False)
    _append_case(64, 2, 32, [(3, 40), (0, 20)], seed=2, drop=(39, 58, 59))


def test_append_many_tokens():
    """Enough tokens for the launch's larger unit of work."""
    _append_case(64, 1, 64, [(5, 1700), (0, 1500), (17, 1400)] + [(9, 1)] * 20, seed=9)


def test_append_zeros_tiny_huge_and_not_finite():
    def tweak(x, heads):
        x[0:16] = 0                                          # a block of zeros
        x[16:32] *= 1e-30                                    # far below the smallest scale
        x[32:48] *= 1e30
        x[48, 0, 0] = 3.3895e38                              # the largest bf16
        x[64, 2 * heads, 3] = math.nan                       # key of head 0
        x[65, 3 * heads + 1, 5] = math.inf                   # value of head 1
        x[66, 2 * heads + 1, 0] = -math.inf
        x[80:96, 2 * heads, 0] = math.nan                    # a whole block of tokens of head 0

    _append_case(128, 2, 16, [(0, 120)], seed=4, tweak=tweak)
    _append_case(64, 2, 64, [(5, 120)], seed=5, tweak=tweak)


def test_append_grows_the_scale_of_a_block():
    """Token by token with growing rows: held bytes are rescaled at every step."""
    V = _v()
    rng = np.random.default_rng(6)
    heads, d, pt = 2, 128, 32
    g = V.make_cache_geom(1, heads, heads, d, 2, pt, 2)
    kc, ks = _pool(rng, 2, heads, pt, d)
    vc, vs = _pool(rng, 2, heads, pt, d)
    host = [_values(kc), _values(vc), ks.double().cpu().numpy(), vs.double().cpu().numpy()]
    for t in range(20):
        x = _bf16(rng, (1, 2 * heads, d), std=2.0 ** rng.integers(-6, 7))
        host = C.append(x[:, :heads].double().numpy(), x[:, heads:].double().numpy(), [32 + t], *host)
        x = x.to(DEV)
        V.vattn_cache_append(g, x[:, :heads], x[:, heads:], ints([32 + t]), kc, vc, ks, vs)
    for got, w in zip((_values(kc), _values(vc), ks.double().cpu().numpy(), vs.double().cpu().numpy()), host):
        np.testing.assert_array_equal(got, w)


def test_append_skips_slots_outside_the_pool():
    V = _v()
    rng = np.random.default_rng(7)
    kc, ks = _pool(rng, 2, 1, 16, 128)
    vc, vs = _pool(rng, 2, 1, 16, 128)
    was = _bytes_of(kc).clone()
    x = _bf16(rng, (4, 1, 128)).to(DEV)
    g = V.make_cache_geom(1, 1, 1, 128, 2, 16, 2)
    V.vattn_cache_append(g, x, x, ints([-1, -5, -1, -2 ** 31]), kc, vc, ks, vs)       # skipped
    _status_ok(V)
    V.vattn_cache_append(g, x, x, ints([32, -5, 2 ** 31 - 1, -2 ** 31]), kc, vc, ks, vs)
    assert V.vattn_get_status() == V.binding.VATTN_ERR_DEVICE_BOUNDS
    assert torch.equal(was, _bytes_of(kc))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Fwd:
    """A cache with streams of given (kv length, new tokens), and queries."""

    def __init__(self, d, kv_heads, group, pt, steps, frame=0, window=0, seed=0, q_std=1.0, extra_rows=3, spread=(-9, -5)):
        self.V = _v()
        rng = np.random.default_rng(seed)
        self.d, self.pt, self.steps, self.frame, self.window = d, pt, steps, frame, window
        self.kv_heads, self.group, self.qh = kv_heads, group, kv_heads * group
        counts = [-(-length // pt) for length, _ in steps]
        self.width = max(1, max(counts)) + 1
        self.pages = sum(counts) + 2
        order = list(rng.permutation(self.pages))
        self.table = np.full((len(steps), self.width), -1)
        for s, c in enumerate(counts):
            self.table[s, :c] = [order.pop() for _ in range(c)]
        self.kc, self.ks = _pool(rng, self.pages, kv_heads, pt, d, *spread)
        self.vc, self.vs = _pool(rng, self.pages, kv_heads, pt, d, *spread)
        # rows behind a stream's last token and unlisted pages hold whatever was there: NaN bytes and scales
        for s, (length, _) in enumerate(steps):
            if length % pt:
                page, row = self.table[s, length // pt], length % pt
                for c in (self.kc, self.vc):
                    _bytes_of(c)[page, :, row:] = 0x7f
                for sc in (self.ks, self.vs):
                    sc[page, :, -(-row // 16):] = math.nan
        for page in order:
            for c, sc in ((self.kc, self.ks), (self.vc, self.vs)):
                _bytes_of(c)[page] = 0xff
                sc[page] = math.nan
        self.n = sum(n for _, n in steps)
        self.rows = self.n + extra_rows
        self.qkv = (_bf16(rng, (self.rows, self.qh + 2, d), q_std)).to(DEV)
        self.q = self.qkv[:, 1:1 + self.qh]
        self.starts = np.cumsum([0] + [n for _, n in steps])
        self.scale = 1 / math.sqrt(d)
        self.dev = dict(starts=ints(self.starts), lens=ints([x for x, _ in steps]), table=ints(self.table))
        self.max_new = max([n for _, n in steps])
        self.geom = self.V.make_cache_geom(len(steps), self.qh, kv_heads, d, self.pages, pt, self.width, frame, window)

    def outputs(self):
        o = torch.full((self.rows, self.qh, self.d), 7.5, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((self.rows, self.qh), 7.5, dtype=torch.float32, device=DEV)
        need = self.V.vattn_cache_workspace_size(self.geom, self.rows, self.max_new)
        self.guard = torch.full((need + 512,), 0xff, dtype=torch.uint8, device=DEV)   # NaN patterns inside, canaries around
        return o, lse, self.guard[256:256 + need]

    def call(self, o, lse, ws, stream=None, max_new=None):
        self.V.vattn_cache_fwd(self.geom, self.q, self.dev["starts"], self.dev["lens"], self.dev["table"], self.kc, self.vc,
                               self.ks, self.vs, self.scale, max_new or self.max_new, o, lse, ws, stream=stream)

    def run(self):
        o, lse, ws = self.outputs()
        self.call(o, lse, ws)
        _status_ok(self.V)
        assert (self.guard[:256] == 0xff).all() and (self.guard[256 + ws.numel():] == 0xff).all()
        return o, lse

    def reference(self, s):
        """(o, lse, a, delta, vmax) of stream s."""
        length, n = self.steps[s]
        q = self.q[self.starts[s]:self.starts[s + 1]].double().cpu().numpy()
        k = C.stream_rows(self.kc_host, self.ks_host, self.table[s], length)
        v = C.stream_rows(self.vc_host, self.vs_host, self.table[s], length)
        mask = C.seen(self.frame, self.window, length, n)
        o, lse, a = C.attend(q, k, v, mask, self.scale)
        kmax = np.abs(k).sum(-1).max(initial=0.0)
        delta = 2.0 ** -16 * self.scale * np.abs(q).max(-1, initial=0.0) * kmax
        return o, lse, a, delta, np.abs(v).max(initial=0.0)

    def check(self, o, lse):
        self.kc_host, self.vc_host = _values(self.kc), _values(self.vc)
        self.ks_host, self.vs_host = self.ks.double().cpu().numpy(), self.vs.double().cpu().numpy()
        og, lg = o.double().cpu().numpy(), lse.double().cpu().numpy()
        for s in range(len(self.steps)):
            a0, a1 = self.starts[s], self.starts[s + 1]
            ro, rl, a, delta, vmax = self.reference(s)
            go, gl = og[a0:a1], lg[a0:a1]
            empty = np.isinf(rl)
            assert np.array_equal(np.isneginf(gl), empty), s
            assert (go[empty] == 0).all(), s
            assert np.isfinite(go).all(), s
            bar = 2.0 ** -8 * np.abs(ro) + (2.0 ** -10 + 2 * delta[..., None]) * a + 2.0 ** -20 * vmax
            worst = (np.abs(go - ro) - bar).max(initial=-1.0)
            assert worst <= 0, (s, worst, np.abs(go - ro).max())
            f = ~empty
            lbar = delta + 2.0 ** -18 * (1 + np.abs(np.where(f, rl, 0)))
            assert (np.abs(gl[f] - rl[f]) <= lbar[f]).all(), (s, np.abs(gl[f] - rl[f]).max())
        assert (og[self.n:] == 7.5).all() and (lg[self.n:] == 7.5).all()      # rows behind the last stream


def _check(**kw):
    f = Fwd(**kw)
    f.check(*f.run())
    return f


TOKENS = [
    [(1, 1)], [(16, 1)], [(17, 1)], [(127, 1)], [(128, 1)], [(129, 1)], [(1000, 1)],
    [(300, 1), (1, 1), (0, 0), (77, 1), (513, 1)],
    [(5, 0), (0, 0), (40, 1)],
    [(i * 37 % 411 + 1, 1) for i in range(40)],
]


@pytest.mark.parametrize("steps", TOKENS, ids=range(len(TOKENS)))
@pytest.mark.parametrize("d,kv_heads,group,pt", [(128, 2, 1, 16), (128, 1, 7, 64), (64, 3, 2, 32), (64, 1, 16, 128)])
def test_single_tokens(d, kv_heads, group, pt, steps):
    _check(d=d, kv_heads=kv_heads, group=group, pt=pt, steps=steps, seed=pt + group)


@pytest.mark.parametrize("d,group,n", [(128, 1, 1), (64, 3, 2), (128, 5, 3), (64, 1, 16)])
@pytest.mark.parametrize("length", [4000, 4400, 30000])
def test_one_head_over_many_keys(d, group, n, length):
    """One kv head whose keys all thread blocks share: few and many partial results."""
    f = Fwd(d=d, kv_heads=1, group=group, pt=128, steps=[(length, n)], frame=1, seed=31)
    f.check(*f.run())


def test_many_streams():
    """More streams than a thread block has threads, most of them short, some idle."""
    steps = [(i * 53 % 90, 1 if i % 7 and i * 53 % 90 else 0) for i in range(700)] + [(3000, 1), (1, 1), (700, 1)]
    _check(d=64, kv_heads=2, group=1, pt=16, steps=steps, seed=30)


FEW = [
    ([(9, 5)], 1, 0), ([(200, 8), (31, 1), (8, 8), (130, 3)], 1, 0), ([(257, 4), (63, 7)], 0, 0),
    ([(100, 6), (333, 8)], 4, 2), ([(3, 8), (0, 3), (2, 2)], 1, 0), ([(500, 5), (90, 5)], 7, 1), ([(300, 3)], 1, 40),
]


@pytest.mark.parametrize("case", FEW, ids=range(len(FEW)))
@pytest.mark.parametrize("d,kv_heads,group,pt", [(128, 2, 2, 16), (64, 2, 1, 64), (128, 1, 3, 128), (64, 1, 5, 32)])
def test_few_tokens(d, kv_heads, group, pt, case):
    steps, frame, window = case
    _check(d=d, kv_heads=kv_heads, group=group, pt=pt, steps=steps, frame=frame, window=window, seed=pt)


MANY = [
    ([(128, 128)], 0, 0), ([(129, 129)], 1, 0), ([(300, 17), (40, 40), (513, 131)], 1, 0),
    ([(700, 200), (64, 33), (0, 0), (256, 256)], 0, 0), ([(640, 260), (100, 100)], 50, 2),
    ([(30, 70), (0, 20), (200, 140)], 16, 0), ([(520, 150)], 1, 100), ([(900, 64)], 300, 1), ([(260, 130)], 128, 1),
]


@pytest.mark.parametrize("case", MANY, ids=range(len(MANY)))
@pytest.mark.parametrize("d,kv_heads,group,pt", [(128, 1, 1, 64), (64, 2, 1, 16), (128, 2, 3, 128), (64, 1, 2, 32),
                                                 (128, 1, 2, 16)])
def test_many_tokens(d, kv_heads, group, pt, case):
    steps, frame, window = case
    _check(d=d, kv_heads=kv_heads, group=group, pt=pt, steps=steps, frame=frame, window=window, seed=pt + 1)


@pytest.mark.parametrize("steps", [[(700, 1), (90, 1)], [(300, 9)], [(400, 200)]], ids=["one", "few", "many"])
def test_sharp_scores_and_scales_of_every_size(steps):
    """Scores up to several hundred, and scales 2^60 apart."""
    _check(d=128, kv_heads=2, group=2, pt=32, steps=steps, seed=1, q_std=20.0)
    _check(d=64, kv_heads=1, group=1, pt=16, steps=steps, seed=2, q_std=1e-4, spread=(-12, 10))
    f = Fwd(d=128, kv_heads=1, group=2, pt=64, steps=steps, seed=3)
    f.vs *= torch.exp2(torch.randint(-30, 31, f.vs.shape, device=DEV).float())
    f.check(*f.run())


@pytest.mark.parametrize("steps", [[(200, 1), (90, 1)], [(130, 9)], [(300, 150)]], ids=["one", "few", "many"])
def test_queries_of_every_size(steps):
    """Zero rows, rows of tiny and of huge values, and rows that mix them."""
    f = Fwd(d=128, kv_heads=1, group=2, pt=32, steps=steps, seed=4)
    f.q[0, 0] = 0
    f.q[0, 1] *= 2.0 ** -100
    f.q[1, 0, 5:] *= 2.0 ** -20
    f.q[1, 1, :3] *= 2.0 ** -130
    f.check(*f.run())


@pytest.mark.parametrize("frame", [0, 1, 40])
@pytest.mark.parametrize("n", [1, 6, 140])
def test_a_token_that_is_not_finite_spoils_only_who_sees_it(n, frame):
    f = Fwd(d=128, kv_heads=2, group=1, pt=32, steps=[(300, n), (200, n)], frame=frame, seed=5)
    page, row = int(f.table[0, 298 // 32]), 298 % 32
    _bytes_of(f.kc)[page, 1, row] = 0x7f                     # as vattn_cache_append stores it
    _bytes_of(f.vc)[page, 1, row] = 0
    f.q[f.starts[1], 0, 3] = math.nan
    o, lse = f.run()
    bad = torch.zeros((f.rows, 2), dtype=torch.bool, device=DEV)
    bad[:n, 1] = torch.from_numpy(C.seen(frame, 0, 300, n)[:, 298]).to(DEV)
    bad[f.starts[1], 0] = True
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    assert torch.equal(torch.isnan(lse), bad)
    # everyone else: as with that token's row made harmless
    _bytes_of(f.kc)[page, 1, row] = 0
    f.q[f.starts[1], 0, 3] = 0
    f.check(*f.run())


@pytest.mark.parametrize("n", [1, 7, 150])
def test_bad_indices_are_reported_and_left_alone(n):
    """A page id, a length or a token range that cannot be: nothing outside is
    read or written, the status says so, other streams are as ever."""
    V = _v()
    for what in ("page", "page-", "length", "start", "count"):
        f = Fwd(d=128, kv_heads=1, group=2, pt=16, steps=[(300, n), (200, n)], seed=6)
        o, lse, ws = f.outputs()
        ok = [x.clone() for x in f.run()]
        if what == "page":
            f.dev["table"][1, 3] = f.pages
        elif what == "page-":
            f.dev["table"][1, 0] = -1
        elif what == "length":
            f.dev["lens"][1] = f.width * 16 + 1
        elif what == "start":
            f.dev["starts"][2] = f.rows + 40
        elif what == "count" and n > 1:
            f.max_new = n - 1                                # promised fewer than there are
        else:
            continue
        f.call(o, lse, ws)
        assert V.vattn_get_status() == V.binding.VATTN_ERR_DEVICE_BOUNDS, what
        assert (f.guard[:256] == 0xff).all() and (f.guard[256 + ws.numel():] == 0xff).all()
        if what != "count":
            assert torch.equal(o[:n], ok[0][:n]) and torch.equal(lse[:n], ok[1][:n]), what
        if what in ("page", "page-"):
            assert (o[f.n:] == 7.5).all()


@pytest.mark.parametrize("steps", [[(900, 1), (300, 1)], [(400, 6)], [(600, 170)]], ids=["one", "few", "many"])
def test_the_same_bits_every_time_without_lse_and_on_another_stream(steps):
    f = Fwd(d=128, kv_heads=2, group=2, pt=64, steps=steps, frame=0, seed=8)
    o, lse = f.run()
    for _ in range(3):
        o2, lse2 = f.run()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, _, ws = f.outputs()
    f.call(o3, None, ws)
    assert torch.equal(o, o3)
    side = torch.cuda.Stream()
    o4, lse4, ws = f.outputs()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f.call(o4, lse4, ws)
    side.synchronize()
    assert torch.equal(o, o4) and torch.equal(lse, lse4)
    # a larger promise than needed picks another kernel or grid, not another result
    f.max_new = f.rows
    o5, lse5 = f.run()
    f.check(o5, lse5)


def test_two_calls_at_once_with_a_workspace_each():
    fs = [Fwd(d=128, kv_heads=4, group=1, pt=64, steps=[(1500 + 100 * i, 1)], seed=20 + i) for i in range(3)]
    want = [f.run() for f in fs]
    streams = [torch.cuda.Stream() for _ in fs]
    outs = [f.outputs() for f in fs]
    torch.cuda.synchronize()
    for _ in range(10):
        for f, st, (o, lse, ws) in zip(fs, streams, outs):
            with torch.cuda.stream(st):
                f.call(o, lse, ws)
    torch.cuda.synchronize()
    for (o, lse, _), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_offsets_past_32_bits():
    """A pool larger than 2^32 bytes whose last pages are the ones in use."""
    V = _v()
    rng = np.random.default_rng(9)
    heads, d, pt = 24, 128, 128
    pages = (2 ** 32 // (heads * pt * d)) + 40
    kc, vc = (torch.zeros((pages, heads, pt, d), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones((pages, heads, pt // 16), device=DEV) for _ in range(2))
    table = ints([[pages - 1, pages - 3, 0, pages - 2]])
    slots = [int(table[0, p // pt]) * pt + p % pt for p in range(450)]
    x = _bf16(rng, (450, 3 * heads, d)).to(DEV)
    g = V.make_cache_geom(1, heads, heads, d, pages, pt, 4)
    V.vattn_cache_append(g, x[:, heads:2 * heads], x[:, 2 * heads:], ints(slots), kc, vc, ks, vs)
    for n in (1, 12, 150):
        o = torch.empty((n, heads, d), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((n, heads), device=DEV)
        ws = torch.empty(V.vattn_cache_workspace_size(g, n, n), dtype=torch.uint8, device=DEV)
        V.vattn_cache_fwd(g, x[450 - n:, :heads], ints([0, n]), ints([450]), table, kc, vc, ks, vs, 0.1, n, o, lse, ws)
        _status_ok(V)
        idx = table[0].long()
        small = [c[idx].float().double().cpu().numpy() for c in (kc, vc)]
        sc = [s[idx].double().cpu().numpy() for s in (ks, vs)]
        k, v = (C.stream_rows(c, s, [0, 1, 2, 3], 450) for c, s in zip(small, sc))
        q = x[450 - n:, :heads].double().cpu().numpy()
        ro, rl, a = C.attend(q, k, v, np.ones((n, 450), dtype=bool), 0.1)
        delta = 2.0 ** -16 * 0.1 * np.abs(q).max() * np.abs(k).sum(-1).max()
        bar = 2.0 ** -8 * np.abs(ro) + (2.0 ** -10 + 2 * delta) * a + 2.0 ** -20 * np.abs(v).max()
        assert (np.abs(o.double().cpu().numpy() - ro) <= bar).all()
        assert (np.abs(lse.double().cpu().numpy() - rl) <= delta + 2.0 ** -18 * (1 + np.abs(rl))).all()


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------

class Serve:
    """Plan, append, attend: one step on device buffers that stay where they are."""

    def __init__(self, frame=0, window=0, streams=4, pt=32, d=128, kv_heads=2, group=2, pages=60, width=24, max_tokens=160):
        self.V = V = _v()
        self.frame, self.window, self.qh, self.kv_heads, self.d, self.pt = frame, window, kv_heads * group, kv_heads, d, pt
        self.max_tokens, self.streams = max_tokens, streams
        self.geom = V.make_cache_geom(streams, self.qh, kv_heads, d, pages, pt, width, frame, window)
        self.lens = torch.zeros(streams, dtype=torch.int32, device=DEV)
        self.table = torch.full((streams, width), -1, dtype=torch.int32, device=DEV)
        self.free = torch.arange(pages, dtype=torch.int32, device=DEV)
        self.n_free = ints([pages])
        self.starts, self.slots = torch.zeros(streams + 1, dtype=torch.int32, device=DEV), torch.zeros(
            max_tokens, dtype=torch.int32, device=DEV)
        self.result = torch.zeros(4, dtype=torch.int32, device=DEV)
        self.kc, self.vc = (torch.full((pages, kv_heads, pt, d), 0x7f, dtype=torch.uint8, device=DEV) for _ in range(2))
        self.ks, self.vs = (torch.full((pages, kv_heads, pt // 16), math.nan, device=DEV) for _ in range(2))
        self.new = torch.zeros(streams, dtype=torch.int32, device=DEV)
        self.qkv = torch.zeros((max_tokens, self.qh + 2 * kv_heads, d), dtype=torch.bfloat16, device=DEV)
        self.o = torch.zeros((max_tokens, self.qh, d), dtype=torch.bfloat16, device=DEV)
        self.lse = torch.zeros((max_tokens, self.qh), device=DEV)
        self.ws = None
        self.history = [[] for _ in range(streams)]

    def inputs(self, new, rng):
        """This step's counts and projections, on the device and in the history."""
        x = _bf16(rng, (sum(max(n, 0) for n in new), self.qkv.shape[1], self.d))
        self.new.copy_(ints(new))
        self.qkv[:len(x)].copy_(x)
        t = 0
        for s, n in enumerate(new):
            if n < 0:
                self.history[s] = []
            for i in range(max(n, 0)):
                self.history[s].append(x[t + i].double().numpy())
            t += max(n, 0)
        return x

    def step(self, max_new, rows=None):
        V, qh, kvh = self.V, self.qh, self.kv_heads
        rows = rows or self.max_tokens
        if self.ws is None or self.ws.numel() < V.vattn_cache_workspace_size(self.geom, rows, max_new):
            self.ws = torch.empty(V.vattn_cache_workspace_size(self.geom, rows, max_new), dtype=torch.uint8, device=DEV)
        V.vattn_cache_plan(self.geom, self.new, self.lens, self.table, self.free, self.n_free, self.lens, self.n_free,
                           self.starts, self.slots, self.result)
        x = self.qkv[:rows]
        V.vattn_cache_append(self.geom, x[:, qh:qh + kvh], x[:, qh + kvh:], self.slots, self.kc, self.vc, self.ks, self.vs)
        V.vattn_cache_fwd(self.geom, x[:, :qh], self.starts, self.lens, self.table, self.kc, self.vc, self.ks, self.vs,
                          0.125, max_new, self.o[:rows], self.lse[:rows], self.ws)

    def check(self, new):
        """Against attention over the exact history, with the cache's rounding as the bar:
        e4m3 keeps 2^-4 of a value; a block's smaller rows lose no more than 2^-10 of its
        largest value beyond that."""
        t = 0
        for s, n in enumerate(new):
            n = max(n, 0)
            if n:
                h = np.stack(self.history[s])
                q, k, v = h[-n:, :self.qh], h[:, self.qh:self.qh + self.kv_heads], h[:, self.qh + self.kv_heads:]
                mask = C.seen(self.frame, self.window, len(h), n)
                ro, rl, a = C.attend(q, k, v, mask, 0.125)
                # scores: rms 2^-4 / sqrt(3) * |q_c k_c| over the channels, six of them; weights move by that factor
                kq = np.sqrt(np.einsum("nhd,lgd->nhlg", q ** 2, k ** 2).max((2, 3)))
                ds = 6 * 0.125 * 2.0 ** -4 / math.sqrt(3) * kq
                bar = 2.0 ** -8 * np.abs(ro) + (2.0 ** -4 + 2 * np.expm1(ds)[..., None]) * a + 2.0 ** -10 * 4
                go, gl = (x[t:t + n].double().cpu().numpy() for x in (self.o, self.lse))
                assert (np.abs(go - ro) <= bar).all()
                assert (np.abs(gl - rl) <= ds + 1e-3).all()
            t += n


@pytest.mark.parametrize("frame,window", [(0, 0), (1, 0), (8, 2)])
def test_generation_step_by_step(frame, window):
    """Prompts, single tokens, a stream that ends and one that takes its place,
    each step against attention over the exact history."""
    rng = np.random.default_rng(11)
    s = Serve(frame, window)
    for new in ([70, 40, 0, 16], [1, 1, 33, 1], [1, 1, 1, 1], [-1, 5, 8, 0], [20, 1, 1, 1], [1, 1, 1, 1], [0, 0, 0, -1],
                [1, 1, 1, 100], [1] * 4):
        s.inputs(new, rng)
        s.step(max(new + [1]))
        assert s.result[0] == 0
        s.check(new)
    _status_ok(s.V)


def test_a_refused_plan_makes_the_step_a_no_op():
    rng = np.random.default_rng(12)
    s = Serve(pages=8, width=24)
    s.inputs([80, 80, 0, 0], rng)
    s.step(80)
    assert s.result[0] == 0
    was = [x.clone() for x in (s.kc, s.vc, s.lens, s.table, s.n_free)]
    s.o.fill_(7.5)
    s.new.copy_(ints([100, 1, 1, 1]))
    s.step(100)
    assert s.result[0] == s.V.VATTN_PLAN_NO_PAGES
    for a, b in zip(was, (s.kc, s.vc, s.lens, s.table, s.n_free)):
        assert torch.equal(a, b)
    assert (s.o == 7.5).all()
    _status_ok(s.V)


def test_a_captured_step_is_replayed():
    """One step captured, replayed with new inputs: state moves on in place,
    and every replay equals the eager step on a copy."""
    rng = np.random.default_rng(13)
    s, e = Serve(max_tokens=8), Serve(max_tokens=8)
    steps = [[2, 1, 3, 1], [1, 1, 1, 1], [1, 0, 1, 2], [-1, 1, 1, 1], [4, 1, 1, 1]]
    x = s.inputs(steps[0], rng)
    e.new.copy_(s.new)
    e.qkv.copy_(s.qkv)
    s.step(4)                                   # first call: allocations, addresses
    e.step(4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step(4)
    for new in steps[1:]:
        x = s.inputs(new, rng)
        e.new.copy_(s.new)
        e.qkv[:len(x)].copy_(s.qkv[:len(x)])
        graph.replay()
        e.step(4)
        n = len(x)
        assert s.result[0] == 0
        for a, b in ((s.o[:n], e.o[:n]), (s.lse[:n], e.lse[:n]), (s.kc, e.kc), (s.lens, e.lens), (s.table, e.table)):
            assert torch.equal(a, b)
        s.check(new)
    del graph
    _status_ok(s.V)


def test_bounded_waits_run_out():
    """The load warp's first arrival withheld: the kernel gives up, reports it
    and leaves the device usable."""
    V = _v()
    f = Fwd(d=128, kv_heads=1, group=2, pt=64, steps=[(400, 200)], seed=15)
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


@pytest.mark.parametrize("streams,top", [(3, 3000), (700, 9), (40, 150), (1500, 2)])
def test_plan_with_slots_of_many_tokens(streams, top):
    """More slots than the planning block lists itself."""
    rng = random.Random(streams)
    p = Planner(streams, 32, 200, 3000, 4500 + streams)
    for _ in range(4):
        new = [rng.choice([-1, 0, 1, rng.randrange(top), top // 2]) for _ in range(streams)]
        if p.step(new):
            assert p.step([-1] * streams) == 0
    _status_ok(p.V)


def test_steps_captured_after_copies_and_across_streams():
    """The launches depend on whatever is ahead of them in the stream: a copy, a
    memset, another stream's work joined by an event, captured or not."""
    f = Fwd(d=128, kv_heads=2, group=2, pt=32, steps=[(700, 1), (90, 1)], seed=16)
    m = Fwd(d=64, kv_heads=2, group=1, pt=32, steps=[(400, 150)], seed=17)
    want = [x.clone() for x in f.run()], [x.clone() for x in m.run()]
    src = [x.q.clone() for x in (f, m)]
    lens = f.dev["lens"].clone()
    (o, lse, ws), (o2, lse2, ws2) = f.outputs(), m.outputs()
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        f.q.copy_(src[0])                                  # a kernel or a copy, then ours
        f.dev["lens"].copy_(lens)                          # device-to-device copy
        f.call(o, lse, ws)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            m.q.copy_(src[1])
            ws2.zero_()
            m.call(o2, lse2, ws2)
        f.call(o, lse, ws)
        main.wait_stream(side)
        m.call(o2, lse2, ws2)                              # after both streams

    def check():
        torch.cuda.synchronize()
        for got, ref in zip((o, lse, o2, lse2), (*want[0], *want[1])):
            assert torch.equal(got, ref)

    step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for x in (f, m):
            x.q.zero_()
        f.dev["lens"].fill_(1)
        o.fill_(7.5)                                       # rows behind the last stream are not written
        o2.fill_(7.5)
        graph.replay()
        check()
    del graph
    _status_ok(f.V)
