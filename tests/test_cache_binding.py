"""What the binding of the cache calls takes and refuses before it calls the library."""
import pytest
import torch

from test_cache import FakeTensor, FakeLib, _geom


@pytest.fixture
def B(monkeypatch):
    import video_dit_local_b200.binding as B
    monkeypatch.setattr(B, "lib", FakeLib())
    monkeypatch.setattr(B, "_current_stream", lambda s, dev: None)
    return B


def test_one_head_may_have_any_stride(B):
    """[tokens, 1, d] with dense rows is dense whatever the stride of its only head: a transposed [1, tokens, d]."""
    g, t = _geom(B, q_heads=1, kv_heads=1), FakeTensor
    for x in (torch.zeros(1, 5, 64).transpose(0, 1), torch.zeros(5, 3, 64)[:, 1:2], torch.zeros(5, 64)[:, None]):
        kv = dict(shape=tuple(x.shape), stride=list(x.stride()))
        B.vattn_cache_append(g, t(**kv), t(**kv), t((5,)), t(), t(), t(), t())
        assert B.lib.calls[-1][1][2] == B.lib.calls[-1][1][4] == x.stride(0)
        B.vattn_cache_fwd(g, t(**kv), t(), t(), t(), t(), t(), t(), t(), 0.1, 3, t(), t(), t((777,)))
        assert B.lib.calls[-1][1][2] == x.stride(0)
    with pytest.raises(ValueError, match="contiguous"):        # two heads are not
        kv = dict(shape=(5, 2, 64), stride=[64, 320, 1])
        B.vattn_cache_append(_geom(B), t(**kv), t(**kv), t((5,)), t(), t(), t(), t())
    with pytest.raises(ValueError, match="contiguous"):
        kv = dict(shape=(5, 1, 64), stride=[64, 1, 5])
        B.vattn_cache_append(g, t(**kv), t(**kv), t((5,)), t(), t(), t(), t())


@pytest.mark.gpu
def test_one_head_transposed_equals_the_dense_one():
    import video_dit_local_b200 as V
    gen = torch.Generator(device="cuda").manual_seed(3)
    g = V.make_cache_geom(1, 1, 1, 128, 4, 16, 4)
    i32 = dict(dtype=torch.int32, device="cuda")
    slots = torch.arange(40, **i32)
    x = torch.randn((3, 1, 40, 128), generator=gen, device="cuda").bfloat16()
    got = []
    for q, k, v in (x.transpose(1, 2), x.transpose(1, 2).contiguous()):
        kc, vc = (torch.zeros((4, 1, 16, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros((4, 1, 1), device="cuda") for _ in range(2))
        V.vattn_cache_append(g, k, v, slots, kc, vc, ks, vs)
        o = torch.zeros((40, 1, 128), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(V.vattn_cache_workspace_size(g, 40, 40), dtype=torch.uint8, device="cuda")
        V.vattn_cache_fwd(g, q, torch.tensor([0, 40], **i32), torch.tensor([40], **i32), torch.arange(4, **i32)[None], kc, vc,
                          ks, vs, 0.1, 40, o, None, ws)
        assert V.vattn_get_status() == 0
        got.append((kc, vc, ks, vs, o))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][4].abs().sum() > 0


class Typed(FakeTensor):
    """A fake tensor that has a type."""

    def __init__(self, shape, dtype=torch.int32, stride=None, **kw):
        super().__init__(shape, stride, **kw)
        self.dtype = dtype
        self.nbytes = self.numel() * dtype.itemsize


def _arrays(**change):
    """The arguments of the three calls for a pool of 10 pages of 16 tokens, 2 kv heads of 64, 2 streams, 4 query heads."""
    bf, f8, f32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32
    a = dict(new=((2,), torch.int32), lens=((2,), torch.int32), table=((2, 4), torch.int32), free=((10,), torch.int32),
             n_free=((1,), torch.int32), lens_out=((2,), torch.int32), n_free_out=((1,), torch.int32),
             starts=((3,), torch.int32), slots=((5,), torch.int32), result=((4,), torch.int32),
             k=((5, 2, 64), bf), v=((5, 2, 64), bf), q=((5, 4, 64), bf), kc=((10, 2, 16, 64), f8), vc=((10, 2, 16, 64), f8),
             ks=((10, 2, 1), f32), vs=((10, 2, 1), f32), o=((5, 4, 64), bf), lse=((5, 4), f32), ws=((640,), torch.uint8))
    a.update(change)
    return {k: Typed(*v) if isinstance(v, tuple) else v for k, v in a.items()}


def _calls(B, a, max_tokens=None, ws_bytes=0):
    g = _geom(B)
    plan = [a[k] for k in ("new", "lens", "table", "free", "n_free", "lens_out", "n_free_out", "starts", "slots", "result")]
    pool = [a[k] for k in ("kc", "vc", "ks", "vs")]
    return dict(
        plan=lambda: B.vattn_cache_plan(g, *plan, max_tokens=max_tokens),
        append=lambda: B.vattn_cache_append(g, a["k"], a["v"], a["slots"], *pool),
        fwd=lambda: B.vattn_cache_fwd(g, a["q"], a["starts"], a["lens"], a["table"], *pool, 0.1, 3, a["o"], a["lse"], a["ws"],
                                      ws_bytes))


def test_arrays_that_fit_pass(B):
    for f in _calls(B, _arrays()).values():
        f()
    # larger ones than needed, bytes as uint8, no lse, raw addresses
    a = _arrays(table=((2, 8), torch.int32), kc=((11, 2, 16, 64), torch.uint8), o=((9, 4, 64), torch.bfloat16), lse=None,
                free=((12,), torch.int32), slots=((9,), torch.int32), vs=4096, lens=4096)
    for f in _calls(B, a).values():
        f()
    assert len(B.lib.calls) == 6


@pytest.mark.parametrize("call,change", [
    (call, {name: bad}) for call, name, bads in [
        ("plan", "new", [((1,), torch.int32), ((2,), torch.int64)]),
        ("plan", "lens", [((1,), torch.int32), ((2,), torch.int64), ((2,), torch.float32)]),
        ("plan", "table", [((2, 3), torch.int32), ((1, 4), torch.int32)]),
        ("plan", "free", [((9,), torch.int32)]),
        ("plan", "n_free", [((0,), torch.int32), ((1,), torch.int64)]),
        ("plan", "lens_out", [((1,), torch.int32)]),
        ("plan", "n_free_out", [((0,), torch.int32)]),
        ("plan", "starts", [((2,), torch.int32)]),
        ("plan", "slots", [((5,), torch.int64)]),
        ("plan", "result", [((3,), torch.int32)]),
        ("append", "k", [((5, 2, 64), torch.float16), ((5, 2, 64), torch.float32), ((5, 1, 64), torch.bfloat16),
                         ((5, 2, 128), torch.bfloat16), ((5, 128), torch.bfloat16)]),
        ("append", "v", [((5, 2, 64), torch.float16), ((5, 3, 64), torch.bfloat16), ((4, 2, 64), torch.bfloat16)]),
        ("append", "slots", [((5,), torch.int64), ((4,), torch.int32)]),
        ("append", "kc", [((9, 2, 16, 64), torch.float8_e4m3fn), ((10, 2, 16, 64), torch.bfloat16),
                          ((10, 2, 16, 64), torch.float8_e5m2), ((10, 2, 16, 64), torch.int8)]),
        ("append", "vc", [((10, 1, 16, 64), torch.uint8)]),
        ("append", "ks", [((9, 2, 1), torch.float32), ((10, 2, 1), torch.bfloat16)]),
        ("append", "vs", [((10, 1, 1), torch.float32)]),
        ("fwd", "q", [((5, 4, 64), torch.float16), ((5, 4, 64), torch.float32), ((5, 2, 64), torch.bfloat16),
                      ((5, 4, 128), torch.bfloat16)]),
        ("fwd", "starts", [((2,), torch.int32), ((3,), torch.int64)]),
        ("fwd", "lens", [((1,), torch.int32)]),
        ("fwd", "table", [((2, 3), torch.int32)]),
        ("fwd", "kc", [((9, 2, 16, 64), torch.float8_e4m3fn)]),
        ("fwd", "vc", [((10, 2, 8, 64), torch.float8_e4m3fn)]),
        ("fwd", "ks", [((9, 2, 1), torch.float32)]),
        ("fwd", "vs", [((10, 2, 1), torch.float64)]),
        ("fwd", "o", [((4, 4, 64), torch.bfloat16), ((5, 4, 64), torch.float16), ((5, 2, 64), torch.bfloat16)]),
        ("fwd", "lse", [((4, 4), torch.float32), ((5, 4), torch.float64), ((5, 4), torch.bfloat16)]),
    ] for bad in bads], ids=lambda x: str(x) if isinstance(x, str) else f"{[*x]}{[*x.values()]}")
def test_arrays_that_do_not_fit_are_refused(B, call, change):
    name = next(iter(change))
    with pytest.raises(ValueError, match="the call needs|the geometry says|slots"):
        _calls(B, _arrays(**change))[call]()
    assert not B.lib.calls, name


def test_sizes_that_the_tensors_do_not_have_are_refused(B):
    with pytest.raises(ValueError, match="slots"):
        _calls(B, _arrays(), max_tokens=6)["plan"]()
    with pytest.raises(ValueError, match="ws_bytes"):
        _calls(B, _arrays(), ws_bytes=641)["fwd"]()
    with pytest.raises(ValueError, match="workspace"):
        _calls(B, _arrays(ws=Typed((640,), torch.uint8, device=1)))["fwd"]()
    assert not B.lib.calls
    _calls(B, _arrays(), max_tokens=4)["plan"]()
    _calls(B, _arrays(), ws_bytes=600)["fwd"]()
    assert [args[-2] for name, args in B.lib.calls if name == "vattn_cache_fwd"] == [600]


@pytest.mark.gpu
def test_real_tensors_that_do_not_fit_are_refused():
    """As above on the GPU: nothing is launched."""
    import video_dit_local_b200 as V
    g = V.make_cache_geom(2, 4, 2, 64, 10, 16, 4)
    a = {k: torch.zeros(x.shape, dtype=x.dtype, device="cuda") for k, x in _arrays().items()}
    size = V.vattn_cache_workspace_size(g, 5, 3)
    a["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    pool = a["kc"], a["vc"], a["ks"], a["vs"]

    def fwd(**kw):
        b = dict(a, **kw)
        V.vattn_cache_fwd(g, b["q"], b["starts"], b["lens"], b["table"], *pool, 0.1, 3, b["o"], b["lse"], b["ws"])

    fwd()
    wide = torch.zeros((5, 9, 64), dtype=torch.bfloat16, device="cuda")
    fwd(q=wide[:, 2:6])
    for bad in (dict(q=wide[:, 2:4]), dict(q=wide[:, 2:6].half()), dict(o=a["o"][:4]), dict(lse=a["lse"].double()),
                dict(lens=a["lens"].long()), dict(starts=a["starts"][:2]), dict(table=a["table"].cpu())):
        with pytest.raises(ValueError):
            fwd(**bad)
    with pytest.raises(ValueError, match="kcache"):
        V.vattn_cache_append(g, a["k"], a["v"], a["slots"], a["kc"][:9], *pool[1:])
    assert V.vattn_get_status() == 0
