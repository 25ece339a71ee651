"""Page ids outside the pool: the plan refuses the step before it hands one out
or writes into one (the definition on CPU, the kernel on the GPU)."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as C

PT, WIDTH, PAGES = 16, 6, 12
BAD = [-1, PAGES, -2 ** 31, 2 ** 31 - 1]


def _state(lens):
    table = np.full((len(lens), WIDTH), -1)
    ids = list(range(PAGES))
    for s, n in enumerate(lens):
        for j in range(-(-n // PT)):
            table[s, j] = ids.pop(0)
    free = np.array(ids + [-1] * (PAGES - len(ids)))
    return dict(lens=list(lens), table=table, free=free, n_free=len(ids))


def _bad_states(bad):
    """(new tokens, state) of steps that meet `bad`."""
    st = _state([20, 32, 0])
    st["free"][st["n_free"] - 2] = bad                  # the second page that the step pops
    yield [16, 0, 16], st
    st = _state([20, 32, 0])
    st["free"][0] = bad                                 # popped last, of all eight free pages
    yield [44, 32, 64], st
    st = _state([20, 32, 0])
    st["free"][st["n_free"] - 1] = bad                  # popped after a stream's two pages are
    yield [-1, 16, 48], st
    st = _state([20, 32, 0])
    st["table"][0, 1] = bad                             # partly filled
    yield [1, 0, 0], st
    st = _state([20, 32, 0])
    st["table"][0, 1] = bad
    yield [30, 1, 1], st
    st = _state([20, 32, 0])
    st["table"][1, 0] = bad                             # given back
    yield [0, -1, 1], st


def _good_states(bad):
    """(new tokens, state) of steps that `bad` does not concern."""
    st = _state([20, 32, 0])
    st["free"][0] = bad                                 # not popped yet
    yield [5, 1, 16], st
    st = _state([20, 32, 0])
    st["free"][st["n_free"] - 1] = bad                  # below the two pages that serve the step
    yield [-1, 16, 16], st
    st = _state([20, 32, 0])
    st["table"][0, 1] = bad                             # of a stream that does not grow
    yield [0, 1, 1], st
    st = _state([20, 32, 0])
    st["table"][1, 2] = bad                             # listed by nobody: the step puts a page there
    yield [0, 1, 1], st
    st = _state([20, 32, 0])
    st["table"][1, 1] = bad                             # full: not written again
    yield [0, 4, 0], st


def _plan(new, st, max_tokens=200):
    return C.plan(PT, WIDTH, PAGES, new, st["lens"], st["table"], st["free"], st["n_free"], max_tokens)


@pytest.mark.parametrize("bad", BAD)
def test_the_definition_refuses_page_ids_that_cannot_be(bad):
    for new, st in _bad_states(bad):
        code, lens, table, _, n_free, starts, slots, _ = _plan(new, st)
        assert code == 4 and lens == st["lens"] and n_free == st["n_free"]
        assert np.array_equal(table, st["table"]) and set(starts) == {0} and set(slots) == {-1}
    for new, st in _good_states(bad):
        code, _, _, _, _, starts, slots, _ = _plan(new, st)
        assert code == 0 and all(x >= 0 for x in slots[:starts[-1]])


@pytest.mark.gpu
@pytest.mark.parametrize("max_tokens", [200, 5000])      # slots listed by the planning block, and by the second kernel
@pytest.mark.parametrize("bad", BAD)
def test_the_plan_refuses_page_ids_that_cannot_be(bad, max_tokens):
    import video_dit_local_b200 as V

    def ints(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    geom = V.make_cache_geom(3, 1, 1, 128, PAGES, PT, WIDTH)
    for new, st in (*_bad_states(bad), *_good_states(bad)):
        lens, table, free, n_free = ints(st["lens"]), ints(st["table"]), ints(st["free"]), ints([st["n_free"]])
        starts, slots, result = ints([7] * 4), ints([7] * max_tokens), ints([7] * 4)
        V.vattn_cache_plan(geom, ints(new), lens, table, free, n_free, lens, n_free, starts, slots, result)
        code, w_lens, w_table, w_free, w_n, w_starts, w_slots, w_result = _plan(new, st, max_tokens)
        assert result.tolist() == w_result and lens.tolist() == w_lens and n_free.tolist() == [w_n]
        assert starts.tolist() == w_starts and slots.tolist() == w_slots
        assert np.array_equal(table.cpu().numpy(), w_table)
        assert np.array_equal(free.cpu().numpy()[:w_n], w_free[:w_n])
        assert V.vattn_get_status() == 0
