"""A workspace sized for the longest step serves every shorter one."""
import math
import random

import pytest
import torch

STEPS = [1, 2, 3, 7, 8, 9, 16, 17, 40, 64, 65, 128, 129, 200, 256, 257, 500, 1024, 1500, 3840, 9000, 17280, 60000]


def _geom(V, streams, kv_heads, group, d=128, page_tokens=64, width=1024):
    return V.make_cache_geom(streams, kv_heads * group, kv_heads, d, 3000, page_tokens, width, 1)


@pytest.mark.parametrize("width", [3, 60, 1024])
@pytest.mark.parametrize("streams,kv_heads,group", [(1, 1, 1), (1, 24, 1), (1, 3, 7), (1, 150, 1), (2, 8, 2), (4, 24, 1),
                                                    (6, 8, 40), (48, 4, 6), (700, 2, 1), (1, 2, 300)])
def test_the_size_never_falls(streams, kv_heads, group, width):
    import video_dit_local_b200 as V
    g = _geom(V, streams, kv_heads, group, width=width)
    sizes = [V.vattn_cache_workspace_size(g, 1 << 20, n) for n in STEPS]
    assert sizes == sorted(sizes)
    assert [V.vattn_cache_workspace_size(g, n, 1 << 20) for n in STEPS] == sizes        # max_new > n_tokens counts as n_tokens
    if group <= 16:
        assert sizes[0] == V.vattn_cache_workspace_size(_geom(V, 2, 1, 1), 1, 1)        # single tokens: of one size
    assert sizes[-1] < 1 << 28                                                          # what splits leave is bounded


def test_nothing_needs_nothing():
    import video_dit_local_b200 as V
    assert V.vattn_cache_workspace_size(_geom(V, 0, 2, 1), 5, 5) == 0
    assert V.vattn_cache_workspace_size(_geom(V, 2, 2, 1), 5, 0) == 0
    assert V.vattn_cache_workspace_size(_geom(V, 2, 2, 1), 0, 5) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("streams,kv_heads,group", [(4, 24, 1), (1, 5, 3), (3, 2, 20)])
def test_one_workspace_serves_every_step(streams, kv_heads, group, d):
    """Steps of every length with the longest one's workspace: as with their own."""
    import video_dit_local_b200 as V
    gen = torch.Generator(device="cuda").manual_seed(d + group)
    width, pt, pages = 24, 64, 40
    g = V.make_cache_geom(streams, kv_heads * group, kv_heads, d, pages, pt, width, 1)
    steps = [n for n in STEPS if n <= 1500]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c = (torch.randn((2, pages, kv_heads, pt, d), generator=gen, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.full((2, pages, kv_heads, pt // 16), 2.0 ** -7, device="cuda")
    table = torch.randint(0, pages, (streams, width), generator=gen, device="cuda").to(torch.int32)
    lens = ints([random.Random(i).randrange(pt, width * pt) for i in range(streams)])
    size = V.vattn_cache_workspace_size(g, steps[-1] * streams, steps[-1])
    guard = torch.empty(size + 512, dtype=torch.uint8, device="cuda")
    for n in steps:
        q = torch.randn((n * streams, kv_heads * group, d), generator=gen, device="cuda").bfloat16()
        starts = ints([n * i for i in range(streams + 1)])
        got = []
        for fill in (0xff, 0x3f):
            guard.fill_(fill)
            o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
            V.vattn_cache_fwd(g, q, starts, lens, table, c[0], c[1], s[0], s[1], 1 / math.sqrt(d), n, o, lse,
                              guard[256:256 + size])
            assert V.vattn_get_status() == 0
            assert (guard[:256] == fill).all() and (guard[256 + size:] == fill).all()
            got.append((o, lse))
        assert not torch.isnan(got[0][0]).any()
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
