"""Calls of more than 2^32 lanes are refused before anything is enqueued (without a
GPU, an attempt to enqueue would show as another error)."""
import ctypes

import parameter_layout_collectives_amd as tide
from parameter_layout_collectives_amd._lib import lib
from test_blocks_host import E_UNSUPPORTED, err

P = ctypes.c_void_p
A = 1 << 47                        # addresses that are never dereferenced, far apart


def at(i):
    return P(A + (i << 56))


def test_linear_refuses_before_it_quantises():
    m, n, k = 1 << 29, 1 << 12, 128
    st = lib().tide_block_linear(at(0), m, k, at(1), at(2), n, at(3), 0x20, at(4), 1 << 50, None)
    assert st == E_UNSUPPORTED and "2^32 lanes" in err()
    assert lib().tide_block_workspace(3, m, n, k, 0x20) == -1
    st = lib().tide_block_mm(at(0), at(1), m, at(2), at(3), n, k, at(4), 0x20, None, 0, None)
    assert st == E_UNSUPPORTED and "2^32 lanes" in err()


def test_unshard_refuses_before_its_first_launch():
    """A first launch's worth of small matrices, then one that no launch can take."""
    plan = tide.Plan([(1 + i % 7, 100 + i) for i in range(300)] + [(1 << 30, 300)], 4096)
    bp = tide.BlockPlan(plan)
    params = (P * 301)(*[A + (1 << 56) + (i << 30) for i in range(301)])
    st = lib().tide_block_unshard(bp.handle, at(0), params, 0x20, None)
    assert st == E_UNSUPPORTED and "2^32 lanes" in err()
