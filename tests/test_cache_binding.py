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
