"""Slots outside the pool in a ring or a table: reported when they are moved, not only when a token lies in them."""
import numpy as np
import pytest
import torch

import sparse_kv_cache_decode_gb300 as K

pytestmark = pytest.mark.gpu
BAD_INDEX = 7
N_SLOTS, BS, NB = 40, 16, 12


def i32(x):
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int64).to(torch.int32).cuda()


@pytest.fixture
def tables():
    k = torch.zeros((1, N_SLOTS, 1, BS, 64), dtype=torch.bfloat16, device="cuda")
    pool = K.Pool(K.make_pool_config(1, N_SLOTS, 1, 1, 64, BS, NB * BS, 3, 512), k, torch.zeros_like(k))
    return K.BlockTables.empty(pool, 3)


@pytest.mark.parametrize("bad", [N_SLOTS, -1, (1 << 31) - 1, -(1 << 31)])
@pytest.mark.parametrize("at", [0, 4, 9])
def test_a_bad_slot_off_the_ring(tables, bad, at):
    tables.ring[at] = bad
    tables.reserve(i32([64, 0, 96]))                    # the first ten slots
    assert tables.pool.poll_error() == BAD_INDEX and tables.pool.poll_error() == 0
    want = list(range(10))
    want[at] = bad
    assert tables.n_held.tolist() == [4, 0, 6] and tables.ring_state.tolist() == [10, 30, 0]
    assert tables.block2slot[0, :4].tolist() + tables.block2slot[2, :6].tolist() == want


def test_a_bad_slot_that_stays_in_the_ring_is_not_looked_at(tables):
    tables.ring[10] = N_SLOTS
    tables.reserve(i32([64, 0, 96]))
    assert tables.pool.poll_error() == 0


@pytest.mark.parametrize("bad", [N_SLOTS, -1])
@pytest.mark.parametrize("to", ["ring", "row"])
@pytest.mark.parametrize("at", [1, 3])
def test_a_bad_slot_given_back(tables, bad, to, at):
    tables.reserve(i32([64, 0, 0]))
    tables.block2slot[0, at] = bad
    if to == "row":                                     # handed over in the same call: the ring is empty
        tables.reserve(i32([64, 192, 192]))
        assert tables.pool.poll_error() == 0
        tables.ring_state.copy_(i32([0, 0, 0]))
        tables.n_held.copy_(i32([4, 0, 0]))
        tables.reserve(i32([0, 64, 0]))
        assert tables.block2slot[1, :4].tolist() == [bad if i == at else i for i in range(4)]
    else:
        tables.reserve(i32([0, 0, 0]))
        assert tables.ring.tolist()[:4] == [bad if i == at else i for i in range(4)] and tables.ring_state.tolist() == [4, 40, 0]
    assert tables.pool.poll_error() == BAD_INDEX


def test_tokens_of_bad_slots_have_no_place(tables):
    tables.ring[1], tables.ring[6] = -7, N_SLOTS
    place, pos = torch.full((6,), 99, dtype=torch.int64, device="cuda"), i32([99] * 6)
    tables.reserve(i32([18, 80, 0]), i32([0, 3, 6, 6]), place, pos)
    assert tables.pool.poll_error() == BAD_INDEX
    assert place.tolist() == [15, -1, -1, -1, -1, -1] and pos.tolist() == [15, 16, 17, 77, 78, 79]
