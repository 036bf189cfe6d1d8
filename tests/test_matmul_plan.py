"""What ssd_matmul_i8 chooses, without a GPU: the sizes of the GPU tests reach every kernel, and no choice can leave two
clusters waiting for each other's tensor memory."""
import random

import pytest

import int8_quant_b200 as iq
from tests import matmul_sizes as S

SMS = 148                                # of a B200
SM_SMEM, CTA_SMEM, CTA_RESERVED = 228 * 1024, 227 * 1024, 1024
TMEM = 512                               # columns of an SM


def plan(T, K, N):
    return iq.ssd_matmul_i8_plan(T, K, N, SMS)


def test_the_tested_sizes_reach_every_kernel_and_split():
    assert all(plan(*a).pair for a in S.PAIRS)
    assert {a[2] % 8 for a in S.PAIRS} == set(range(8))
    assert {a[2] % 256 for a in S.PAIRS} >= {1, 2, 7, 63, 65, 127, 129, 255}
    for (bn, split), a in S.FEW.items():
        p = plan(*a)
        assert (p.pair, p.tile_tokens, p.split) == (0, bn, split), a
    assert set(S.FEW) == {(bn, s) for bn in (16, 32, 64, 128) for s in (1, 2, 4, 8)}
    for T, N, pair in S.EXTREME:
        assert plan(T, S.LONGEST_K, N).pair == pair, (T, N)
    assert {(N % 8 == 0) for _, N, pair in S.EXTREME if pair} == {True, False}


def _random_sizes(n, seed):
    rng = random.Random(seed)
    for _ in range(n):
        yield round(20000 ** rng.random()), 16 * round(8191 ** rng.random()), round(30000 ** rng.random())


def test_choices_fit_an_sm():
    for T, K, N in _random_sizes(20000, 1):
        p = plan(T, K, N)
        slices = -(-K // 128)
        assert p.smem_bytes <= CTA_SMEM and p.tmem_columns <= TMEM
        assert p.stages >= 1 and 1 <= p.split <= min(8, slices)
        if p.pair:
            assert T > 64 and p.ctas % 2 == 0 and p.ctas <= SMS
        else:
            tiles = -(-T // p.tile_tokens) * -(-N // p.tile_channels)
            assert p.ctas == tiles * p.split and p.tile_channels % 8 == 0 and 64 <= p.tile_channels <= 128
            # a stage belongs to one of two issuing warps, so their number is even once stages are used again
            per_rank = -(-slices // p.split)
            assert p.stages == per_rank or (p.stages < per_rank and (p.tile_tokens == 128 or p.stages % 2 == 0))


def test_clusters_of_several_calls_cannot_starve_each_other_of_tensor_memory():
    """A CTA of a cluster waits for the others, and taking tensor memory waits until enough is free.  Calls of several
    streams may share SMs: so the CTAs of any mixture of clusters that fit an SM's shared memory together have to find
    their columns there.  (CTAs that wait for no other always end, and free theirs.)"""
    least = {}                           # columns of a cluster's CTA: the least shared memory that it takes

    def see(T, K, N):
        p = plan(T, K, N)
        if p.pair or p.split > 1:
            least[p.tmem_columns] = min(least.get(p.tmem_columns, CTA_SMEM), p.smem_bytes)

    for a in _random_sizes(60000, 2):
        see(*a)
    for slices in range(1, 24):          # the shortest splits take the least
        for T in (1, 16, 17, 32, 33, 64, 65, 128, 129, 256, 300, 512):
            for N in (*range(1, 130, 16), *range(128, 9000, 128)):
                see(T, 128 * slices - 16, N)
                see(T, 128 * slices - 112, N)
    assert set(least) == {32, 64, 128, 512}
    best = [0] * (SM_SMEM // 1024 + 1)   # columns of the worst mixture in so many KB (unbounded knapsack)
    for kb in range(len(best)):
        for cols, smem in least.items():
            size = (smem + CTA_RESERVED) // 1024
            if size <= kb:
                best[kb] = max(best[kb], best[kb - size] + cols)
    assert max(best) <= TMEM, (best[-1], least)


@pytest.mark.parametrize("args,status", [((-1, 64, 8, SMS), 1), ((4, 0, 8, SMS), 1), ((4, 64, 0, SMS), 1),
                                         ((4, 64, 8, 1), 1), ((4, 40, 8, SMS), 2), ((4, 131072, 8, SMS), 2),
                                         ((2 ** 30 + 1, 64, 8, SMS), 2)])
def test_plan_refuses_what_the_product_refuses(args, status):
    with pytest.raises(iq.SsdError) as err:
        iq.ssd_matmul_i8_plan(*args)
    assert err.value.status == status


def test_plan_of_no_tokens():
    p = iq.ssd_matmul_i8_plan(0, 64, 8)
    assert (p.pair, p.ctas, p.split) == (0, 0, 0)
    assert iq.library().ssd_matmul_i8_plan(4, 64, 8, SMS, None) == 1
