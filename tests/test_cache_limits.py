"""The largest counts that the cache calls take, and what is refused past them."""
import pytest
import torch

TOP = 2 ** 31 - 1


class Rows:
    """Stands in for a [tokens, heads, 64] tensor on a machine without a GPU."""

    def __init__(self, n, heads):
        self.shape = (n, heads, 64)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 16

    def numel(self):
        return self.shape[0]

    def stride(self):
        return self.shape[1] * 64, 64, 1


def test_counts_past_the_limits_are_refused_before_a_launch():
    import video_dit_local_b200 as V

    def geom(streams, heads, group=1):
        return V.make_cache_geom(streams, heads * group, heads, 64, 4, 16, 4)

    def append(n, heads):
        x = Rows(n, heads)
        V.vattn_cache_append(geom(1, heads), x, x, x, 16, 16, 16, 16, stream=0)

    def fwd(streams, heads, max_new):
        V.vattn_cache_fwd(geom(streams, heads), Rows(TOP, heads), 16, 16, 16, 16, 16, 16, 16, 0.1, max_new, 16, 16, 16,
                          1 << 40, stream=0)

    refused = [
        lambda: append(2 ** 30, 16), lambda: append(TOP, 65535),
        lambda: fwd(60000, 30000, TOP), lambda: fwd(65535, 1, TOP), lambda: fwd(2 ** 8, 2 ** 7, 2 ** 24),
        lambda: V.vattn_cache_workspace_size(geom(60000, 30000), TOP, TOP),
        lambda: V.vattn_cache_workspace_size(geom(2 ** 8, 2 ** 7), TOP, 2 ** 24),
    ]
    for i, f in enumerate(refused):
        with pytest.raises(V.VattnError) as e:
            f()
        assert e.value.code == V.binding.VATTN_ERR_UNSUPPORTED, (i, str(e.value))
    assert V.vattn_cache_workspace_size(geom(2 ** 8, 2 ** 7), TOP, 2 ** 24 - 256) > 0
    assert V.vattn_cache_workspace_size(geom(2, 2), TOP, TOP) > 0


def test_a_scale_whose_base_2_form_is_infinite_is_refused():
    import video_dit_local_b200 as V
    g = V.make_cache_geom(1, 1, 1, 64, 4, 16, 4)
    for scale in (2.4e38, 3.4e38):          # finite; times log2(e) past the largest float
        with pytest.raises(V.VattnError) as e:
            V.vattn_cache_fwd(g, Rows(5, 1), 16, 16, 16, 16, 16, 16, 16, scale, 3, 16, 16, 16, 1 << 40, stream=0)
        assert e.value.code == V.binding.VATTN_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("max_tokens", [TOP, TOP - 254, TOP - 255, TOP - 256])
def test_plan_lists_as_many_slots_as_there_can_be(max_tokens):
    import video_dit_local_b200 as V
    i32 = dict(dtype=torch.int32, device="cuda")
    geom = V.make_cache_geom(2, 1, 1, 128, 9, 16, 8)
    lens, table, n_free = torch.tensor([20, 0], **i32), torch.full((2, 8), -1, **i32), torch.tensor([7], **i32)
    table[0, 0], table[0, 1] = 7, 8
    free, starts, result = torch.arange(9, **i32), torch.empty(3, **i32), torch.empty(4, **i32)
    slots = torch.full((max_tokens + 64,), -7, **i32)
    V.vattn_cache_plan(geom, torch.tensor([3, 18], **i32), lens, table, free, n_free, lens, n_free, starts, slots, result,
                       max_tokens=max_tokens)
    assert V.vattn_get_status() == 0 and result.tolist() == [0, 21, 5, 23]
    assert slots[:21].tolist() == [8 * 16 + 4, 8 * 16 + 5, 8 * 16 + 6, *range(96, 112), 80, 81]
    for a in range(21, max_tokens, 1 << 28):
        assert bool((slots[a:min(a + (1 << 28), max_tokens)] == -1).all())
    assert (slots[max_tokens:] == -7).all()
