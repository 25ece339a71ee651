"""Slot lists whose blocks' tokens are not adjacent: refused by the definition
(CPU); the kernel drops the tokens that come back to a block and says so."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as C

# (slots, entries that come back to a block)
LISTS = [
    ([32, -1, 33], [2]),                                        # a skipped entry inside a block
    ([32, 48, 33, 49, 34], [2, 3, 4]),                          # two streams' tokens in turn
    ([36, 37, 37, 38], [2, 3]),                                 # the same slot twice
    ([40, 41, 32, 33, 64], [2, 3]),                             # back to the block's start
    ([33, 32], [1]),                                            # descending
    ([32] + [-1] * 31 + [33, 80], [32]),                        # 32 entries apart
    ([32, 33, 64] + [-1] * 15 + [34, 35, 65, 96], [18, 19, 20]),
    ([5] + list(range(80, 95)) + [6], [16]),                    # the block of another 16 entries
]
GOOD = [[32, 33, 48, 49], [47, 48], [-1, 40, 41, -1, 64, -1], list(range(20, 60)) + [-1] * 40 + list(range(64, 70))]


def _zeros(heads, d, pages=8, pt=16):
    return [np.zeros((pages, heads, pt, d)), np.zeros((pages, heads, pt, d)), np.ones((pages, heads, 1)), np.ones((pages, heads, 1))]


@pytest.mark.parametrize("case", LISTS, ids=range(len(LISTS)))
def test_the_definition_refuses_lists_that_come_back(case):
    slots, _ = case
    x = np.ones((len(slots), 1, 4))
    with pytest.raises(ValueError, match="comes back"):
        C.append(x, x, slots, *_zeros(1, 4))


@pytest.mark.parametrize("slots", GOOD, ids=range(len(GOOD)))
def test_the_definition_takes_adjacent_tokens(slots):
    x = np.ones((len(slots), 1, 4))
    kc, _, _, _ = C.append(x, x, slots, *_zeros(1, 4))
    assert kc[:, 0, :, 0].ravel()[[s for s in slots if s >= 0]].all()


def _append(slots, heads, d, pad=0):
    """The kernel and the definition of `slots` and the entries of it that they are to store."""
    import video_dit_local_b200 as V
    gen = torch.Generator(device="cuda").manual_seed(len(slots))
    pt, pages = 16, 8 + pad
    n = len(slots)
    kv = torch.randn((2, n, heads, d), generator=gen, device="cuda").bfloat16()
    c = (torch.randn((2, pages, heads, pt, d), generator=gen, device="cuda") * 50).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.exp2(torch.randint(-9, -4, (2, pages, heads, 1), generator=gen, device="cuda").float())
    host = [*c.float().double().cpu().numpy(), *s.double().cpu().numpy()]
    geom = V.make_cache_geom(1, heads, heads, d, pages, pt, 1)
    V.vattn_cache_append(geom, kv[0], kv[1], torch.tensor(slots, dtype=torch.int32, device="cuda"), c[0], c[1], s[0], s[1])
    return V.vattn_get_status(), kv.double().cpu().numpy(), host, [*c.float().double().cpu().numpy(), *s.double().cpu().numpy()]


@pytest.mark.gpu
@pytest.mark.parametrize("case", LISTS, ids=range(len(LISTS)))
@pytest.mark.parametrize("heads,d", [(1, 128), (3, 64)])
def test_tokens_that_come_back_to_a_block_are_dropped_and_reported(heads, d, case):
    import video_dit_local_b200 as V
    slots, back = case
    code, kv, host, got = _append(slots, heads, d)
    assert code == V.binding.VATTN_ERR_DEVICE_BOUNDS
    kept = [-1 if i in back else x for i, x in enumerate(slots)]
    for g, w in zip(got, C.append(kv[0], kv[1], kept, *host)):
        np.testing.assert_array_equal(g, w)


@pytest.mark.gpu
@pytest.mark.parametrize("slots", GOOD, ids=range(len(GOOD)))
@pytest.mark.parametrize("heads,d", [(1, 128), (3, 64)])
def test_adjacent_tokens_are_stored(heads, d, slots):
    code, kv, host, got = _append(slots, heads, d)
    assert code == 0
    for g, w in zip(got, C.append(kv[0], kv[1], slots, *host)):
        np.testing.assert_array_equal(g, w)


@pytest.mark.gpu
def test_a_block_come_back_to_in_a_long_list():
    """Enough tokens for the launch's larger unit of work: a warp looks through 16 entries."""
    import video_dit_local_b200 as V
    heads, d, n = 24, 64, 1700
    slots = [-1] * 5 + list(range(n))           # token of slot x: entry x + 5
    slots[805] = slots[806] = -1                # slots 802 .. 815 follow two that the block held before
    slots[413] = -1                             # 409 .. 415 come back, in the warp that takes 400 .. 407
    slots[624] = -1                             # 620 .. 623 come back, in the warp after that of 608 .. 618
    back = [*range(414, 421), *range(625, 629)]
    code, kv, host, got = _append(slots, heads, d, pad=n // 16)
    assert code == V.binding.VATTN_ERR_DEVICE_BOUNDS
    kept = [-1 if i in back else x for i, x in enumerate(slots)]
    for g, w in zip(got, C.append(kv[0], kv[1], kept, *host)):
        np.testing.assert_array_equal(g, w)
