"""The 8-bit key/value cache on CPU: the oracle's pins, the binding's argument
marshalling, and what the entry points refuse before any launch."""
import math
import random

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C


@pytest.fixture(scope="module")
def V():
    import video_dit_local_b200 as V
    return V


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------

def test_e4m3_rounding_is_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.uniform(-0.02, 0.02, 20000), [0.0, 448.0, -448.0]])
    x = x.astype(np.float32)      # torch converts from float32
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(C.round_e4m3(x), want)
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    every = every[np.isfinite(every)]
    assert np.array_equal(C.round_e4m3(every), every)


def test_scale_exponent_is_the_smallest():
    for m in (1e-30, 448 * 2.0 ** -40, 449 * 2.0 ** -40, 1.0, 1.75, 1.7500001, 3.5, 448.0, 450.0, 3e38):
        e = C.scale_exponent(m)
        assert m <= 448 * 2.0 ** e and (e == C.E_MIN or m > 448 * 2.0 ** (e - 1))
    assert C.scale_exponent(0.0) == C.E_MIN


@pytest.mark.parametrize("frame,window", [(0, 0), (1, 0), (3, 0), (4, 2), (1, 5)])
def test_attention_matches_torch_sdpa_with_the_mask(frame, window):
    rng = np.random.default_rng(frame * 10 + window)
    n, length, d = 7, 19, 8
    q, k, v = rng.normal(size=(n, 6, d)), rng.normal(size=(length, 2, d)), rng.normal(size=(length, 2, d))
    mask = C.seen(frame, window, length, n)
    if frame == 1 and window == 0:
        assert np.array_equal(mask, np.tril(np.ones((n, length), dtype=bool), length - n))
    o, lse, _ = C.attend(q, k, v, mask, 0.3)
    tq, tk, tv = (torch.from_numpy(x).transpose(0, 1) for x in (q, k.repeat(3, 1), v.repeat(3, 1)))
    ref = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, attn_mask=torch.from_numpy(mask), scale=0.3)
    np.testing.assert_allclose(o, ref.transpose(0, 1).numpy(), atol=1e-12)
    x = np.einsum("nhd,lhd->hnl", q, k.repeat(3, 1)) * 0.3
    np.testing.assert_allclose(lse.T, np.log(np.where(mask, np.exp(x), 0).sum(-1)), atol=1e-12)


def test_rows_that_see_nothing():
    mask = C.seen(2, 0, 3, 5)             # five new tokens, three left in the cache: positions -2 .. 2
    assert mask.any(1).tolist() == [False, False, True, True, True]
    assert C.seen(2, 1, 8, 3).sum(1).tolist() == [2, 2, 2]
    o, lse, _ = C.attend(np.ones((5, 1, 4)), np.ones((3, 1, 4)), np.ones((3, 1, 4)), mask, 1.0)
    assert (o[:2] == 0).all() and (lse[:2] == -math.inf).all() and np.isfinite(lse[2:]).all()


def test_append_chunk_by_chunk_is_the_whole_up_to_the_scale_it_grew_to():
    """Appending a block in pieces of growing size gives the scale of the whole
    block, and bytes within one rounding of its own."""
    rng = np.random.default_rng(3)
    k = rng.normal(size=(16, 1, 8)) * np.exp2(np.arange(16) / 3)[:, None, None]
    zero = np.zeros((1, 1, 16, 8)), np.zeros((1, 1, 16, 8)), np.zeros((1, 1, 1)), np.zeros((1, 1, 1))
    whole = C.append(k, k, list(range(16)), *zero)
    part = zero
    for a, b in ((0, 1), (1, 4), (4, 9), (9, 16)):
        part = C.append(k[a:b], k[a:b], list(range(a, b)), *part)
    assert np.array_equal(part[2], whole[2])
    np.testing.assert_allclose(part[0], whole[0], rtol=2 ** -3, atol=2 ** -9)


def test_plan_keeps_every_page_in_one_place():
    rng = random.Random(5)
    pt, width, pages, streams = 16, 9, 40, 6
    lens, table = [0] * streams, np.full((streams, width), -1)
    free, n_free = np.arange(pages)[::-1].copy(), pages
    seen_status = set()
    for _ in range(200):
        new = [rng.choice([-1, 0, 1, 1, 17, 40]) for _ in range(streams)]
        st, lens2, table, free, n_free2, starts, slots, res = C.plan(pt, width, pages, new, lens, table, free, n_free, 150)
        seen_status.add(st)
        if st:
            assert lens2 == lens and n_free2 == n_free and set(slots) <= {-1}
            new = [-1] * streams          # start again
            st, lens2, table, free, n_free2, starts, slots, res = C.plan(pt, width, pages, new, lens, table, free, n_free, 150)
            assert st == 0
        lens, n_free = lens2, n_free2
        held = [int(table[s, j]) for s in range(streams) for j in range(-(-lens[s] // pt))]
        assert sorted(held + free[:n_free].tolist()) == list(range(pages))
        real = [x for x in slots if x >= 0]
        assert len(set(real)) == len(real) == starts[-1]
    assert {0, 2} <= seen_status


# ---------------------------------------------------------------------------
# binding and refusals
# ---------------------------------------------------------------------------

class FakeTensor:
    """Stands in for a CUDA tensor on a machine without one."""

    def __init__(self, shape=(4,), stride=None, addr=4096, cuda=True, device=0):
        self.shape, self.addr, self.is_cuda, self.device_ = shape, addr, cuda, device
        self.stride_ = stride or [int(np.prod(shape[i + 1:])) for i in range(len(shape))]

    def data_ptr(self):
        return self.addr

    def is_contiguous(self):
        return True

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return 1

    def stride(self):
        return tuple(self.stride_)

    def get_device(self):
        return self.device_ if self.is_cuda else -1


class FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def B(monkeypatch):
    import video_dit_local_b200.binding as B
    monkeypatch.setattr(B, "lib", FakeLib())
    monkeypatch.setattr(B, "_current_stream", lambda s, dev: None)
    return B


def _geom(V, **kw):
    a = dict(streams=2, q_heads=4, kv_heads=2, head_dim=64, pages=10, page_tokens=16, table_width=4, frame_tokens=0,
             window_frames=0)
    a.update(kw)
    return V.make_cache_geom(**a)


def test_wrappers_pass_the_declared_arguments(B):
    g, t = _geom(B), FakeTensor
    qkv = dict(shape=(5, 4, 64), stride=[512, 64, 1])
    B.vattn_cache_plan(g, *(t() for _ in range(10)))
    B.vattn_cache_append(g, t(**dict(qkv, shape=(5, 2, 64))), t(**dict(qkv, shape=(5, 2, 64))), t((9,)), t(), t(), t(), t())
    B.vattn_cache_fwd(g, t(**qkv), t(), t(), t(), t(), t(), t(), t(), 0.1, 3, t(), t(), t((777,)))
    B.vattn_cache_workspace_size(g, 5, 3)
    got = {name: args for name, args in B.lib.calls}
    assert set(got) == set(B._CACHE_SIGS)
    for name, args in got.items():
        assert len(args) == len(B._CACHE_SIGS[name]), name
    assert got["vattn_cache_plan"][10] == 4                           # max_tokens: the length of slots
    assert got["vattn_cache_append"][2] == got["vattn_cache_append"][4] == 512 and got["vattn_cache_append"][6] == 5
    assert got["vattn_cache_fwd"][2] == 512 and got["vattn_cache_fwd"][11:13] == (5, 3)
    assert got["vattn_cache_fwd"][16] == 777


def test_wrappers_refuse_wrong_tensors(B, monkeypatch):
    g, t = _geom(B), FakeTensor
    kv = dict(shape=(5, 2, 64))
    with pytest.raises(ValueError, match="host tensor"):
        B.vattn_cache_append(g, t(**kv, cuda=False), t(**kv), t((5,)), t(), t(), t(), t())
    with pytest.raises(ValueError, match="contiguous"):
        B.vattn_cache_append(g, t(**kv, stride=[128, 1, 2]), t(**kv), t((5,)), t(), t(), t(), t())
    with pytest.raises(ValueError, match="slots"):
        B.vattn_cache_append(g, t(**kv), t(**kv), t((4,)), t(), t(), t(), t())
    with pytest.raises(ValueError, match="another device"):
        B.vattn_cache_append(g, t(**kv), t(**kv, device=1), t((5,)), t(), t(), t(), t())
    with pytest.raises(ValueError, match="current device"):
        B.vattn_cache_append(g, t(**kv), t(**kv), t((5,)), t(), t(device=1), t(), t())
    with pytest.raises(ValueError, match="host tensor"):
        B.vattn_cache_plan(g, t(), t(), t(), t(cuda=False), *(t() for _ in range(6)))
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        B.vattn_cache_fwd(g, t((5, 4, 64)), *(t() for _ in range(7)), 0.1, 3, t())
    assert not B.lib.calls


def _plan(V, g, **kw):
    a = dict(new=16, lens=16, table=16, free=16, n_free=16, lens_out=16, n_free_out=16, starts=16, slots=16, result=16)
    a.update(kw)
    n = a.pop("max_tokens", 5)
    V.vattn_cache_plan(g, *a.values(), max_tokens=n, stream=0)


class Tok(FakeTensor):
    pass


def _append(V, g, k=None, v=None, slots=None, kc=16, vc=16, ks=16, vs=16):
    kv = dict(shape=(5, 2, 64), addr=16)
    V.vattn_cache_append(g, k or Tok(**kv), v or Tok(**kv), slots or FakeTensor((5,), addr=16), kc, vc, ks, vs, stream=0)


def _fwd(V, g, q=None, scale=0.1, max_new=3, o=16, lse=16, ws=32, ws_bytes=1 << 40, **kw):
    a = dict(starts=16, lens=16, table=16, kc=16, vc=16, ks=16, vs=16)
    a.update(kw)
    V.vattn_cache_fwd(g, q or Tok((5, 4, 64), addr=16), *a.values(), scale, max_new, o, lse, ws, ws_bytes, stream=0)


def test_refusals(V):
    B = V.binding
    UNS, INV, SHP, ALN, WS = (B.VATTN_ERR_UNSUPPORTED, B.VATTN_ERR_INVALID_ARG, B.VATTN_ERR_SHAPE, B.VATTN_ERR_ALIGN,
                              B.VATTN_ERR_WORKSPACE)
    g = _geom(V)
    cases = [(lambda k=k, v=v: _plan(V, _geom(V, **{k: v})), code) for k, v, code in [
        ("streams", -1, INV), ("pages", -1, INV), ("q_heads", 0, INV), ("kv_heads", 0, INV), ("q_heads", 3, SHP),
        ("table_width", 0, INV), ("frame_tokens", -1, INV), ("window_frames", -1, INV), ("window_frames", 2, INV),
        ("head_dim", 96, UNS), ("head_dim", 256, UNS), ("page_tokens", 8, UNS), ("page_tokens", 48, UNS),
        ("page_tokens", 256, UNS), ("q_heads", 65536, UNS), ("streams", 65536, UNS), ("pages", 1 << 27, UNS),
        ("pages", 1 << 60, UNS), ("table_width", 1 << 27, UNS), ("table_width", (1 << 27) - 8, UNS)]]
    cases += [(lambda: _plan(V, _geom(V, streams=65535, kv_heads=65535, q_heads=65535)), UNS),
              (lambda: _plan(V, _geom(V, pages=1 << 26, kv_heads=64, q_heads=64)), UNS),
              (lambda: V.vattn_cache_workspace_size(_geom(V, q_heads=64, kv_heads=1), 1 << 28, 1 << 28), UNS)]
    cases += [(lambda k=k: _plan(V, g, **{k: 0}), INV) for k in
              ("new", "lens", "table", "free", "n_free", "lens_out", "n_free_out", "starts", "slots", "result")]
    cases += [
        (lambda: _plan(V, g, table=18), ALN),
        (lambda: _plan(V, g, max_tokens=-1), INV),
        (lambda: _plan(V, g, max_tokens=1 << 31), UNS),
        (lambda: _append(V, g, k=Tok((5, 2, 64), addr=24)), ALN),
        (lambda: _append(V, g, k=Tok((5, 2, 64), [132, 64, 1], 16)), ALN),
        (lambda: _append(V, g, v=Tok((5, 2, 64), [120, 64, 1], 16)), SHP),
        (lambda: _append(V, g, kc=0), INV),
        (lambda: _append(V, g, vs=24), ALN),
        (lambda: _fwd(V, g, scale=0.0), INV),
        (lambda: _fwd(V, g, scale=-1.0), INV),
        (lambda: _fwd(V, g, scale=math.nan), INV),
        (lambda: _fwd(V, g, scale=math.inf), INV),
        (lambda: _fwd(V, g, max_new=-1), INV),
        (lambda: _fwd(V, _geom(V, pages=0)), INV),
        (lambda: _fwd(V, g, q=Tok((5, 4, 64), [200, 64, 1], 16)), SHP),
        (lambda: _fwd(V, g, q=Tok((5, 4, 64), addr=20)), ALN),
        (lambda: _fwd(V, g, lse=20), ALN),
        (lambda: _fwd(V, g, o=0), INV),
        (lambda: _fwd(V, g, table=0), INV),
        (lambda: _fwd(V, g, kc=0), INV),
        (lambda: V.vattn_cache_workspace_size(g, -1, 1), INV),
        (lambda: V.vattn_cache_workspace_size(g, 1 << 31, 1), UNS),
        (lambda: V.vattn_cache_workspace_size(g, 1, -1), INV),
    ]
    for i, (f, code) in enumerate(cases):
        with pytest.raises(V.VattnError) as e:
            f()
        assert e.value.code == code, (i, str(e.value))


def test_workspace_is_refused_when_short(V):
    g = _geom(V)
    need = V.vattn_cache_workspace_size(g, 5, 3)
    assert need == V.vattn_cache_workspace_size(g, 5, 3)
    if need:
        for kw in (dict(ws=None, ws_bytes=0), dict(ws=32, ws_bytes=need - 1)):
            with pytest.raises(V.VattnError) as e:
                _fwd(V, g, **kw)
            assert e.value.code == V.binding.VATTN_ERR_WORKSPACE
        with pytest.raises(V.VattnError) as e:
            _fwd(V, g, ws=24)
        assert e.value.code == V.binding.VATTN_ERR_ALIGN


def test_nothing_to_do_touches_nothing(V):
    g0 = _geom(V, streams=0)
    _plan(V, g0, **{k: 0 for k in ("new", "lens", "table", "free", "n_free", "lens_out", "n_free_out", "starts",
                                   "slots", "result")})
    empty = Tok((0, 2, 64), addr=0)
    _append(V, _geom(V), k=empty, v=empty)
    _fwd(V, g0, o=0, kc=0)
    _fwd(V, _geom(V), q=Tok((0, 4, 64), addr=0), o=0, kc=0)
    _fwd(V, _geom(V), max_new=0, o=0, kc=0)


def test_constants_match_the_header(V):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "include", "vattn.h")).read()
    found = dict(re.findall(r"(VATTN_PLAN_\w+) = (\d+)", src))
    assert len(found) == 5
    for name, value in found.items():
        assert getattr(V, name) == int(value)
    assert (C.SCALE_TOKENS, C.E_MIN) == (16, -40)
