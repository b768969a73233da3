"""The 4-bit history cache's calls where they go wrong most easily, against the float64 oracle: pages that run
out between requests of all sizes, scores and weights of all sizes, the forms that only large calls take, mixed
batches, and the calls together with the encoder.  Tolerances are those of test_gpu_kv_cache.py unless a test says
otherwise."""
import math

import numpy as np
import pytest
import torch

from oracle import kv_cache as KC
from tests import test_gpu_kv_cache as base
from tests.gpu_util import check_bf16, dev, dev_i32, host, stream
from tests.test_gpu_kv_cache import Cached, R, check_tables, close, run_tables, status  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- pages that run out -----------------------------------------------------------------------------------
@pytest.mark.parametrize("rows", [91, 400])            # one thread a request; tiles of rows
def test_a_request_that_does_not_fit_leaves_the_pages_to_others(R, rows):  # noqa: F811
    got = run_tables(R, None, np.array([20, 70, 1]), 16, np.array([8, 3, 6], np.int32), 10, np.full((3, 5), -1, np.int32), rows)
    assert status(R) == 7
    assert got["kv"].tolist() == [20, 0, 1] and got["off"].tolist() == [0, 20, 90, 91] and got["used"].tolist() == [3]
    assert got["table"][:, :2].tolist() == [[8, 3], [-1, -1], [6, -1]] and (got["table"][:, 2:] == -1).all()
    want = np.full(rows, -1)
    want[:20], want[90] = [*range(128, 144), *range(48, 52)], 96
    assert np.array_equal(got["slots"], want)
    want[:20], want[90] = range(20), 0
    assert np.array_equal(got["pos"], want)


@pytest.mark.parametrize("B,new_top", [(2, 300), (33, 3), (33, 300), (700, 5), (700, 90), (2048, 4), (2048, 60), (2049, 60), (5000, 2), (5000, 60), (20000, 9)])
def test_block_tables_run_out_between_requests_of_all_sizes(R, B, new_top):  # noqa: F811
    """Small requests behind large ones, with little to a lot of the free list there: each takes what the ones in
    front of it left."""
    g = np.random.default_rng(B + new_top)
    page = 16
    new = np.minimum(np.round(np.exp(g.normal(np.log(new_top / 4 + 1), 1.5, B))).astype(np.int64), 40 * new_top)
    past = g.integers(0, 60, B)
    held, after = (past + page - 1) // page, (past + new + page - 1) // page
    order = g.permutation(int(after.sum()) + 5).astype(np.int32)
    table = np.full((B, int(after.max())), -1, np.int32)
    k = 0
    for r in range(B):
        table[r, :held[r]] = order[k:k + held[r]]
        k += held[r]
    need = after - held
    total = int(need.sum())
    new_bad = np.array(new)
    new_bad[g.integers(0, B)] = -3
    for n in sorted({0, 1, int(need.max()) // 2, int(need.max()), total // 10, total // 2, total - 1, total}):
        check_tables(R, past, new if n % 2 else new_bad, page, order[k:k + n], len(order), table, int(new.sum()) + 2)


def test_block_tables_one_request_is_refused_a_turn(R):  # noqa: F811
    """The needs go 1, n, 1, n - 1, 1, n - 2, ..: each large one finds a page too few after the small one before it."""
    B, page = 3000, 16
    new = np.ones(B, np.int64)
    new[1::2] = page * (np.arange(B // 2)[::-1] + 1)
    table = np.full((B, B // 2), -1, np.int32)
    for n in (B // 2, B // 2 + 7, 40):
        check_tables(R, None, new, page, np.arange(n, dtype=np.int32), n, table, int(new.sum()))


def test_block_tables_run_out_far_behind(R):  # noqa: F811
    """More requests than one pass over the sums of their chunks covers: the free list ends far behind, near the
    start, or a page before the last request."""
    B, page = 300000, 16
    g = np.random.default_rng(1)
    new = g.integers(0, 4, B)
    new[g.integers(0, B, 3000)] = 40
    table = np.full((B, 3), -1, np.int32)
    total = int(((new + 15) // 16).sum())
    for n in (total - 1, total - 3000, total // 1000):
        check_tables(R, None, new, page, g.permutation(n).astype(np.int32), n, table, int(new.sum()))


# ---- attention ----------------------------------------------------------------------------------------------------
def fill(c, K, V):
    """Puts K and V [H, tokens, d] of every request's history (the same for all) into the cache of a Cached."""
    for r, n in enumerate(c.lens):
        t = np.arange(n)
        slots = c.table[r, t // c.page].astype(np.int64) * c.page + t % c.page
        c.cache = KC.append(c.cache, c.page, K[:, :n].transpose(1, 0, 2), V[:, :n].transpose(1, 0, 2), slots)
    c.K, c.V = KC.values(c.cache, c.page, c.d)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("counts,lens,share", [([1, 1], [64, 200], 1), ([3, 2], [500, 64], 4), ([20, 9], [128, 65], 1), ([1], [9000], 2),
                                               ([130, 40], [300, 64], 1), ([50], [5000], 2)])
def test_attention_of_equal_values_gives_that_value(R, counts, lens, d, share):  # noqa: F811
    """Every value is 63/32, so every output is, whatever the weights are, as long as their sum is of the weights
    that multiply the values.  One key in 64 has weight 1, the others 1/2 + 1.05 * 2^-9, which bf16 rounds up to
    1/2 + 2^-8: divided by the sum of the unrounded weights the result would be 63/32 * (1 + 2^-8 * 0.93 or more),
    past the middle (63/32 * (1 + 2^-9 * 1.016)) between 63/32 and the next bf16 number.  Sums and products carry
    fp32 errors, far below that."""
    c = Cached(31, counts, lens, 2, share, d, 64)
    n = max(lens)
    K, V = np.zeros((2, n, d)), np.full((2, n, d), 63 / 32)
    K[:, :, 0], K[:, :, 1] = 6, 7                        # element 1 fixes the group's scale at 1
    K[:, ::64, 0] = 7
    fill(c, K, V)
    c.Q = np.zeros_like(c.Q)
    c.Q[:, :, 0] = 1
    got = c.run(R, -math.log(0.5 + 1.05 * 2.0 ** -9), 0)
    assert status(R) == 0 and (got == 63 / 32).all(), np.unique(got)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("counts,lens,share", [([1, 1], [64, 200], 1), ([3, 2], [500, 70], 4), ([20, 9], [128, 65], 1), ([1], [9000], 2),
                                               ([130, 40], [300, 64], 1), ([50], [5000], 2)])
@pytest.mark.parametrize("unit,scale", [(2.0 ** 34, 1.0), (2.0 ** 34, -0.7), (2.0 ** 115, 3.0), (2.0 ** 20, 2.0 ** 100), (1.0, 2.0 ** 126), (1.0, -8e37),
                                        (2.0 ** 11, 0.3), (2.0 ** 118, 0.0), (2.0 ** 118, 1e-40), (2.0 ** 118, 2.5e-37)])
def test_attention_of_scores_of_all_sizes(R, counts, lens, d, share, unit, scale):  # noqa: F811
    """Scores from far above what fp32 tells apart by less than 2^7 to far below one.  A row's queries are 1, 2, .. in element 0,
    keys are whole multiples of `unit` there, so scores are exact in fp32 and the tolerance is the usual one; the last
    three scales make weights between 0.05 and 1 of scores near the largest number."""
    c = Cached(32, counts, lens, 2, share, d, 64)
    g = np.random.default_rng(5)
    n = max(lens)
    K, V = np.zeros((2, n, d)), g.integers(-7, 8, (2, n, d)).astype(np.float64)
    V[:, :, ::32] = 7
    K[:, :, 0], K[:, :, 1] = g.integers(-7, 8, (2, n)) * unit, 7 * unit
    fill(c, K, V)
    c.Q = np.zeros_like(c.Q)
    c.Q[:, :, 0] = 1 + np.arange(c.rows)[:, None] % 4
    got = c.run(R, scale, 0)
    assert status(R) == 0
    close(got, *c.want(np.float64(np.float32(scale)), 0))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("counts,lens,share", [([12, 13], [64, 200], 1), ([3, 2], [500, 70], 4), ([1], [9000], 2), ([130, 40], [300, 64], 1)])
def test_attention_of_scores_far_from_zero(R, counts, lens, d, share):  # noqa: F811
    """Every row's scores have a mean of its own, from 3 to 7000, and differ by halves: exact in fp32 (at most 17 bits), and so
    is a difference of two."""
    c = Cached(33, counts, lens, 2, share, d, 64)
    g = np.random.default_rng(6)
    n = max(lens)
    K, V = np.zeros((2, n, d)), g.integers(-7, 8, (2, n, d)).astype(np.float64)
    V[:, :, ::32] = 7
    K[:, :, 0], K[:, :, 1] = 7, g.integers(-7, 8, (2, n))
    fill(c, K, V)
    c.Q = np.zeros_like(c.Q)
    c.Q[:, :, 0] = 2.0 ** ((np.arange(c.rows)[:, None] + np.arange(2 * share)) % 12)
    c.Q[:, :, 1] = 0.5
    got = c.run(R, 0.5, 0)
    assert status(R) == 0
    close(got, *c.want(0.5, 0))


@pytest.mark.parametrize("at,inside", [("q", 0), ("q", 3840), ("o", 0), ("o", 3840), ("cache", 8960), ("table", 3840), ("kv", 0), ("off", 0)])
def test_attention_refuses_a_workspace_over_its_tensors(R, at, inside):  # noqa: F811
    """The addresses are far apart and of no memory: the call is refused before anything reads them."""
    from request_candidate_sharing_b200 import rocs
    d = rocs.Kv4Desc(16, 16, 1, 32)            # 9216 bytes
    a = {k: (i + 1) << 32 for i, k in enumerate(("q", "o", "cache", "table", "kv", "off"))}
    n = R.rocs_dca_cross_attn_kv4_workspace(d, 8, 1, 8, 1024)
    assert 256 < n < 1 << 32
    for ws in (a[at] + inside, a[at] + inside - n // 256 * 256):          # over the tensor's end, and over its start
        if ws + n <= a[at]:
            continue
        with pytest.raises(rocs.RocsError) as e:
            R.rocs_dca_cross_attn_kv4(d, a["q"], 256, 8, a["cache"], a["table"], 1024, a["kv"], a["off"], 1, 8, 1.0, 0, a["o"], 256, ws, n, stream())
        assert e.value.status == rocs.ROCS_ERR_INVALID_ARG and "the workspace overlaps" in str(e.value)


@pytest.mark.parametrize("rows", [1, 64])
def test_attention_of_a_history_past_a_billion_tokens(R, rows):  # noqa: F811
    """Its pages are three pages over and over, so the result is that of three pages' keys, each weighed by how often it comes.
    A block has up to 2^30 / 444 keys, 16 or more of them in each addition to a sum that may lose 2^-23 of it: 2^-23 * 2^18 of mag
    beside the usual tolerance."""
    from request_candidate_sharing_b200 import rocs
    page, d = 128, 32
    c = Cached(34, [rows], [3 * page], 1, 1, d, page)
    g = np.random.default_rng(1)
    length = 2 ** 30 + 5 * page + 77
    blocks = -(-length // page)
    table = c.table[0, g.choice(3, blocks, p=[0.5, 0.3, 0.2])]
    desc = rocs.Kv4Desc(c.n_pages, page, 1, d)
    q, cache, t = torch.from_numpy(c.Q).to(torch.bfloat16).cuda(), torch.from_numpy(c.cache).cuda(), torch.from_numpy(table).cuda()
    kv, off = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([length], [0, rows]))
    out = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    n = R.rocs_dca_cross_attn_kv4_workspace(desc, 1, 1, rows, blocks)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    R.rocs_dca_cross_attn_kv4(desc, q, d, 1, cache, t, blocks, kv, off, 1, rows, 0.2, 0, out, d, ws, n, stream())
    assert status(R) == 0
    times = np.array([(table[:-1] == p).sum() for p in c.table[0, :3]])[:, None] + (np.arange(page) < 77) * (table[-1] == c.table[0, :3])[:, None]
    assert times.sum() == length
    k, v = (x[c.table[0, :3], 0].reshape(-1, d) for x in (c.K, c.V))
    s = c.Q[:, 0] @ k.T * 0.2
    w = np.exp(s - s.max(-1, keepdims=True)) * times.reshape(-1)
    w /= w.sum(-1, keepdims=True)
    want, mag = w @ v, w @ np.abs(v)
    got = host(out)
    assert (np.abs(got - want) <= 2.0 ** -8 * (mag + np.abs(want)) * (1 + 2.0 ** -8) + (2.0 ** -10 + 2.0 ** -5) * mag).all()
