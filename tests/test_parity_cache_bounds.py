"""Indices that cannot be, with canaries around every array that the call
writes and a copy of every array that it reads: nothing outside is written, the
status says so, other streams are as ever."""
import numpy as np
import pytest
import torch

from test_parity_cache import DEV, Fwd, _bytes_of, _v, ints

pytestmark = pytest.mark.gpu

GUARD = 4096


def _guarded(count, dtype, fill):
    """(whole buffer as bytes, the `count` elements in its middle)."""
    size = count * torch.empty((), dtype=dtype).element_size()
    whole = torch.full((size + 2 * GUARD,), 0xa5, dtype=torch.uint8, device=DEV)
    part = whole[GUARD:GUARD + size].view(dtype)
    part.fill_(fill)
    return whole, part


BAD = {
    "page": lambda f: f.dev["table"][1].__setitem__(3, f.pages),
    "page -1": lambda f: f.dev["table"][1].__setitem__(0, -1),
    "page far": lambda f: f.dev["table"][1].__setitem__(slice(0, 8), ints([2 ** 31 - 1, -2 ** 31] * 4)),
    "every page": lambda f: f.dev["table"][1].fill_(-1),
    "length": lambda f: f.dev["lens"].__setitem__(1, f.width * f.pt + 1),
    "length far": lambda f: f.dev["lens"].__setitem__(1, 2 ** 31 - 1),
    "length negative": lambda f: f.dev["lens"].__setitem__(1, -2 ** 31),
    "start": lambda f: f.dev["starts"].__setitem__(2, f.rows + 40),
    "start far": lambda f: f.dev["starts"].__setitem__(2, 2 ** 31 - 1),
    "start back": lambda f: f.dev["starts"].__setitem__(2, int(f.starts[1]) - 1),
    "start negative": lambda f: f.dev["starts"].__setitem__(2, -2 ** 31),
}


@pytest.mark.parametrize("what", BAD)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 7, 60, 150])
def test_nothing_outside_is_written(n, d, what):
    V = _v()
    f = Fwd(d=d, kv_heads=1, group=2, pt=16, steps=[(300, n), (200, n)], seed=6)
    ok = [x.clone() for x in f.run()]
    BAD[what](f)
    o_all, o = _guarded(f.rows * f.qh * d, torch.bfloat16, 7.5)
    lse_all, lse = _guarded(f.rows * f.qh, torch.float32, 7.5)
    o, lse = o.view(f.rows, f.qh, d), lse.view(f.rows, f.qh)
    ws_all, ws = _guarded(V.vattn_cache_workspace_size(f.geom, f.rows, f.max_new), torch.uint8, 0xff)
    read = [f.qkv, f.kc, f.vc, f.ks, f.vs, *f.dev.values()]
    was = [x.clone() for x in read]
    f.call(o, lse, ws)
    assert V.vattn_get_status() == V.binding.VATTN_ERR_DEVICE_BOUNDS
    for whole in (o_all, lse_all, ws_all):
        assert (whole[:GUARD] == 0xa5).all() and (whole[-GUARD:] == 0xa5).all()
    for a, b in zip(was, read):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(o[:n], ok[0][:n]) and torch.equal(lse[:n], ok[1][:n])      # the first stream
    if "start" not in what:                                                       # rows behind the last stream
        assert (o[f.n:] == 7.5).all() and (lse[f.n:] == 7.5).all()
    got = Fwd(d=d, kv_heads=1, group=2, pt=16, steps=[(300, n), (200, n)], seed=6).run()
    assert torch.equal(got[0], ok[0]) and torch.equal(got[1], ok[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [8, 60, 150])
def test_more_new_tokens_than_promised(n, d):
    V = _v()
    f = Fwd(d=d, kv_heads=1, group=1, pt=16, steps=[(300, n - 1), (200, n)], seed=6)
    ok = [x.clone() for x in f.run()]
    f.max_new = n - 1
    o, lse, ws = f.outputs()
    f.call(o, lse, ws)
    assert V.vattn_get_status() == V.binding.VATTN_ERR_DEVICE_BOUNDS
    assert (f.guard[:256] == 0xff).all() and (f.guard[256 + ws.numel():] == 0xff).all()
    assert (o[f.n:] == 7.5).all() and (lse[f.n:] == 7.5).all()
    f.check(*ok)


@pytest.mark.parametrize("heads,d", [(1, 128), (3, 64)])
def test_append_writes_nothing_outside(heads, d):
    """Slots outside the pool among good ones: the good ones' blocks alone change."""
    V = _v()
    pages, pt = 6, 32
    blocks = pages * heads * pt // 16
    rng = np.random.default_rng(heads)
    arrays = [_guarded(blocks * 16 * d, torch.uint8, 0x11) for _ in range(2)] + [
        _guarded(blocks, torch.float32, 2.0 ** -7) for _ in range(2)]
    slots = [0, 1, 2, pages * pt, 2 ** 31 - 1, -1, pages * pt - 1, -2 ** 31, 2 ** 30, 48, 49]
    x = torch.from_numpy(rng.normal(size=(len(slots), heads, d))).to(torch.bfloat16).to(DEV)
    g = V.make_cache_geom(1, heads, heads, d, pages, pt, 1)
    V.vattn_cache_append(g, x, x, ints(slots), *[a for _, a in arrays])
    assert V.vattn_get_status() == V.binding.VATTN_ERR_DEVICE_BOUNDS
    for whole, _ in arrays:
        assert (whole[:GUARD] == 0xa5).all() and (whole[-GUARD:] == 0xa5).all()
    for _, a in arrays[:2]:
        same = (a.view(pages, heads, pt // 16, 16 * d) == 0x11).all(-1).all(1)
        assert same.tolist() == [[False, True], [True, False]] + [[True, True]] * 3 + [[True, False]]
    assert _bytes_of(arrays[0][1].view(torch.float8_e4m3fn)).view(pages, heads, pt, d)[0, :, :3].ne(0x11).any()
