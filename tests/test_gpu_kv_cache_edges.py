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


# ---- forms that only large calls take ----------------------------------------------------------------------------
@pytest.mark.parametrize("rows,Hq,Hk,d,rot,inter,io", [
    # several items a warp; heads in two units, the second one partly filled; bf16 whole heads, both pairings
    (5003, 12, 3, 32, 32, 0, 1), (5003, 12, 3, 32, 32, 1, 1), (5003, 5, 7, 64, 64, 0, 1), (5003, 5, 7, 64, 64, 1, 1), (2003, 3, 3, 128, 128, 0, 1),
    (2003, 3, 3, 128, 128, 1, 1), (3601, 1, 1, 256, 256, 0, 1), (5003, 17, 0, 16, 16, 1, 1),
    # parts of heads, and fp32
    (5003, 5, 7, 64, 32, 1, 1), (5003, 3, 2, 80, 48, 1, 1), (5003, 5, 7, 64, 64, 1, 0), (5003, 3, 2, 96, 64, 1, 0), (5003, 3, 2, 96, 64, 0, 0),
])
def test_qk_norm_rope_of_many_rows(R, rows, Hq, Hk, d, rot, inter, io):  # noqa: F811
    base.test_qk_norm_rope(R, rows, Hq, Hk, d, rot, inter, io, 1)


@pytest.mark.parametrize("rows,H,page,d", [(30011, 5, 16, 32), (120001, 1, 64, 32), (14209, 8, 128, 32), (30011, 5, 32, 64), (15007, 5, 16, 128)])
def test_append_and_gather_of_many_rows(R, rows, H, page, d):  # noqa: F811
    """Two row sets a warp, with skipped rows and an odd end."""
    base.test_append_and_gather(R, rows, H, page, d)


@pytest.mark.parametrize("B,H,share,d,causal", [
    (300, 8, 1, 32, 0), (300, 8, 1, 32, 1), (700, 5, 1, 32, 0), (250, 8, 2, 64, 1), (450, 5, 1, 128, 0),         # two warps a head
    (1300, 3, 1, 32, 0), (700, 8, 1, 32, 0), (700, 8, 1, 32, 1), (1000, 5, 2, 32, 0), (1000, 5, 1, 64, 1), (800, 6, 1, 128, 0),      # one
    (8200, 3, 1, 32, 0), (8200, 3, 1, 32, 1), (8200, 5, 1, 64, 0),                 # one, past the list
])
def test_attention_of_many_heads_a_block(R, B, H, share, d, causal):  # noqa: F811
    """Few rows of many requests: a block takes several neighbouring heads, the last block of a tile fewer."""
    g = np.random.default_rng(B + H)
    lens = g.integers(0, 300 if B < 8000 else 40, B)
    lens[::7] = g.integers(0, 3, len(lens[::7]))
    c = Cached(35, g.integers(0, 3, B), lens, H, share, d, 16, pad_rows=3)
    got = c.run(R, d ** -0.5, causal)
    assert status(R) == 0
    n = int(c.offsets[-1])
    want, mag = c.want(d ** -0.5, causal)
    close(got[:n], want[:n], mag[:n])
    assert (got[n:] == 9).all()


@pytest.mark.parametrize("counts,pad", [([1] * 480 + [200] * 8, 5), ([0] * 200 + [300, 0, 0, 180, 7] + [0] * 100, 1200), ([1, 1, 700, 1] * 6, 0)])
@pytest.mark.parametrize("d,share", [(32, 1), (64, 2), (128, 1)])
def test_attention_of_mixed_and_padded_batches(R, counts, pad, d, share):  # noqa: F811
    """Single rows and bursts in one call, and a captured step's empty requests and padded rows."""
    g = np.random.default_rng(len(counts))
    c = Cached(36, counts, g.integers(0, 700, len(counts)), 1, share, d, 64, pad_rows=pad)
    got = c.run(R, d ** -0.5, 0)
    assert status(R) == 0
    n = int(c.offsets[-1])
    want, mag = c.want(d ** -0.5, 0)
    close(got[:n], want[:n], mag[:n])
    assert (got[n:] == 9).all()


@pytest.mark.parametrize("q,B,H,lens", [(40, 300, 2, 40), (1, 600, 8, 40), (1, 5, 1, 9000), (3, 40, 1, 5000), (50, 3, 1, 5000)])
def test_attention_offsets_back_and_forth_write_nothing_from_a_list(R, q, B, H, lens):  # noqa: F811
    """Listed and split forms: requests that all claim every row would not fit the list, so none is done."""
    c = Cached(37, [q] * B, [lens] * B if B > 5 else [lens, 0, 70, 0, 300][:B], H, 1, 32, 16)
    off = np.where(np.arange(B + 1) % 2 == 0, 0, c.rows)
    got = c.run(R, 0.2, 0, offsets=off)
    assert status(R) == 5 and (got == 9).all()


@pytest.mark.parametrize("rows", [70, 5003])
@pytest.mark.parametrize("d,rot,inter,io", [(32, 32, 0, 1), (64, 32, 1, 1), (128, 128, 0, 0), (80, 48, 1, 0)])
def test_qk_norm_rope_of_heads_of_all_sizes(R, rows, d, rot, inter, io):  # noqa: F811
    """Heads whose squares leave fp32's range at either end lie beside common ones; eps is 0 or counts only for the smallest."""
    from request_candidate_sharing_b200 import rocs
    g = np.random.default_rng(rows + d)
    dt, H = torch.bfloat16 if io else torch.float32, 3
    size = 2.0 ** np.array([0, 124, -120, 63, -66, 90, -50, 10, 60, -130])
    buf = torch.from_numpy((np.clip(g.normal(size=(rows, H, d)), -6, 6) * size[np.arange(rows * H).reshape(rows, H, 1) % 10]).astype(np.float32)).to(dt)
    x, pos, cs = buf.double().numpy(), g.integers(0, 50, rows), KC.angles(50, rot)
    t, post, cst = buf.reshape(rows, -1).cuda(), dev_i32(pos), torch.from_numpy(cs).cuda()
    for eps in (0.0, 2.0 ** -110):
        out = torch.zeros_like(t)
        desc = rocs.QkDesc(rows, H, 0, d, rot, inter, 50, eps, io)
        R.rocs_qk_norm_rope(desc, t, H * d, None, 0, None, None, cst, post, out, H * d, None, 0, stream())
        assert status(R) == 0
        y, mag = KC.qk_norm_rope(x, None, eps, cs, pos, inter)
        tol = 16 * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(y) if io else 0)
        assert (np.abs(host(out).reshape(rows, H, d) - y) <= tol * (1 + 2.0 ** -8) + 1e-30).all()


# ---- the calls together ----------------------------------------------------------------------------------------------
@pytest.mark.parametrize("B,H,share,d,page", [(4, 2, 2, 64, 16), (3, 2, 1, 32, 64)])
def test_serving_steps_norm_and_rotate_by_their_positions(R, B, H, share, d, page):  # noqa: F811
    """The queries and keys that a step's attention works on, against the oracle's norm and rotation of what was
    handed in, at each event's place in its history."""
    g = np.random.default_rng(40 + B)
    rows, Hq = 96, H * share
    st = base.Step(R, B, H, share, d, page, 8, 60, rows)
    gamma, cs = st.gamma.cpu().numpy(), st.cs.cpu().numpy()
    past = np.zeros(B, int)
    hist = [[] for _ in range(B)]
    for new in (g.integers(10, 25, B), np.ones(B, int), np.array([1, 0, 17] + [3] * (B - 3))):
        x = base.bf16(g.normal(size=(rows, st.width)))
        st.new.copy_(dev_i32(new))
        st.qkv.copy_(x.cuda())
        st.calls()
        assert status(R) == 0
        pos = np.concatenate([p + np.arange(n) for p, n in zip(past, new)] + [np.full(rows - new.sum(), -1)])
        assert np.array_equal(st.pos.cpu().numpy(), pos)
        was, qkv, n = x.double().numpy(), host(st.qkv), int(new.sum())
        for at, heads in ((0, Hq), (Hq * d, H)):
            y, mag = KC.qk_norm_rope(was[:, at:at + heads * d].reshape(rows, heads, d), gamma, 1e-6, cs, pos, 0)
            got = qkv[:, at:at + heads * d].reshape(rows, heads, d)
            tol = (16 * 2.0 ** -24 * mag + 2.0 ** -8 * np.abs(y)) * (1 + 2.0 ** -8)
            assert (np.abs(got - y) <= tol)[:n].all() and (got[n:] == was[n:, at:at + heads * d].reshape(-1, heads, d)).all()
        assert np.array_equal(qkv[:, (Hq + H) * d:], was[:, (Hq + H) * d:])            # the values are not touched
        want, mag = base.reference_step(hist, new, qkv, st.off.cpu().numpy(), H, share, d, page, None, None)
        close(host(st.out)[:n].reshape(n, Hq, d), want, mag)
        past += new
        st.past.copy_(st.kv)
        used = int(st.used.item())
        st.free.copy_(torch.cat([st.free[used:], st.free[:used]]))


def test_serving_step_with_a_refused_request(R):  # noqa: F811
    """A burst finds too few pages: its rows have position -1, it keeps its history, the others are served, and what the causal
    attention writes for it is what the header says, its plain queries against the tokens it holds, shifted."""
    B, H, share, d, page, rows = 3, 2, 1, 32, 16, 96
    g = np.random.default_rng(50)
    st = base.Step(R, B, H, share, d, page, 8, 60, rows)
    hist = [[] for _ in range(B)]
    for new, n_free in (([10, 20, 5], 60), ([3, 40, 12], 1)):
        new = np.array(new)
        x = base.bf16(g.normal(size=(rows, st.width)))
        st.new.copy_(dev_i32(new))
        st.qkv.copy_(x.cuda())
        st.free = st.free[:n_free].contiguous()
        st.calls()
        assert status(R) == (0 if n_free > 1 else 7)
        qkv, off, out = host(st.qkv), st.off.cpu().numpy(), host(st.out).reshape(rows, H, d)
        if n_free > 1:
            want, mag = base.reference_step(hist, new, qkv, off, H, share, d, page, None, None)
            close(out[:35], want, mag)
            used = int(st.used.item())
            st.past.copy_(st.kv)
            st.free = st.free[used:].contiguous()
    assert st.kv.tolist() == [13, 20, 17] and off.tolist() == [0, 3, 43, 55] and st.used.item() == 1
    pos = st.pos.cpu().numpy()
    assert pos[:3].tolist() == [10, 11, 12] and (pos[3:43] == -1).all() and pos[43:55].tolist() == list(range(5, 17)) and (pos[55:] == -1).all()
    assert (qkv[3:43] == x.double().numpy()[3:43]).all()
    # the others, as without it
    served = np.r_[0:3, 43:55]
    want, mag = base.reference_step([hist[0], hist[2]], np.array([3, 12]), qkv[served], np.array([0, 3, 15]), H, share, d, page, None, None)
    close(out[served], want, mag)
    old = np.concatenate(hist[1])
    kv = [KC.dequantize(*KC.quantize(y)).transpose(1, 0, 2)[None] for y in (old[:, H:2 * H], old[:, 2 * H:])]
    want, mag = KC.attention(qkv[3:43, :H * d].reshape(40, H, d), H, *kv, np.zeros((1, 1), int), [20], [0, 40], 20, d ** -0.5, 1)
    close(out[3:43], want, mag)
    assert (out[3:23] == 0).all() and (out[55:] == 9).all()


def test_encoded_histories_in_the_cache(R):  # noqa: F811
    """The encoder's candidate-side keys and values of ragged histories (padded to L rows a request) go to the cache by the slots
    of the block tables, candidates attend to them there, and they come back for the dense attention."""
    import synth
    from request_candidate_sharing_b200 import rocs
    lengths, counts = np.array([37, 64, 1, 50]), np.array([5, 0, 70, 33])
    case = synth.model_cfg4(B_R=4, counts=list(counts))
    a, B, page = case.dca, 4, 16
    L, d, H = a.L, a.d, a.H
    dh = d // H
    assert L >= 64 and dh == 64
    W, x = synth.model_weights(case), synth.model_inputs(case)
    Wd = {k: dev(v, torch.float32 if "ln." in k else torch.bfloat16) for k, v in W.items()}
    desc = rocs.DcaDesc(B, L, d, H, a.layers)
    nb = R.rocs_dca_encode_workspace(desc)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    S, KV = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((a.layers, B, L, d), (a.layers, 4, B, L, d)))
    n_new = dev_i32(lengths)
    R.rocs_dca_encode(desc, dev(x["H"]), [rocs.dca_layer_weights(Wd, l) for l in range(a.layers)], S, KV, ws, nb, stream(), lengths=n_new)
    K, V = KV[-1, 2], KV[-1, 3]
    # slots of the compact rows, laid out by the padded rows' places: -1 past each history's end
    total, n_pages, blocks = int(lengths.sum()), 20, L // page + 1
    table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
    kv, off, used, pos = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in (B, B + 1, 1, total))
    slots = torch.zeros(total, dtype=torch.int64, device="cuda")
    free = torch.randperm(n_pages, generator=torch.Generator().manual_seed(3)).int().cuda()
    R.rocs_kv_block_tables(None, n_new, B, page, free, n_pages, n_pages, table, blocks, kv, off, slots, pos, total, used, None, 0, stream())
    padded = torch.full((B, L), -1, dtype=torch.int64, device="cuda")
    padded[torch.arange(L, device="cuda") < n_new[:, None]] = slots
    cdesc = rocs.Kv4Desc(n_pages, page, H, dh)
    cache = torch.zeros(n_pages, H, KC.record_bytes(page, dh), dtype=torch.uint8, device="cuda")
    R.rocs_kv4_append(cdesc, K, d, V, d, padded, B * L, cache, stream())
    assert status(R) == 0
    real = host(padded.reshape(-1)) >= 0
    want_cache = KC.append(np.zeros(cache.shape, np.uint8), page, host(K).reshape(-1, H, dh)[real], host(V).reshape(-1, H, dh)[real], slots.cpu().numpy())
    assert np.array_equal(cache.cpu().numpy(), want_cache)
    # candidates over the cache
    rows = int(counts.sum())
    Q = base.bf16(np.random.default_rng(8).normal(size=(rows, d)))
    offsets = np.concatenate([[0], np.cumsum(counts)])
    out = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    n = R.rocs_dca_cross_attn_kv4_workspace(cdesc, H, B, rows, blocks)
    aws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    Qd, offd = Q.cuda(), dev_i32(offsets)
    R.rocs_dca_cross_attn_kv4(cdesc, Qd, d, H, cache, table, blocks, kv, offd, B, rows, dh ** -0.5, 0, out, d, aws, n, stream())
    assert status(R) == 0
    want, mag = KC.attention(Q.double().numpy().reshape(rows, H, dh), H, *KC.values(want_cache, page, dh), table.cpu().numpy(), lengths, offsets, page,
                             dh ** -0.5, 0)
    close(host(out).reshape(rows, H, dh), want, mag)
    # and back, for the dense attention over the same values
    Kb, Vb = torch.zeros_like(K), torch.zeros_like(V)
    R.rocs_kv4_gather(cdesc, cache, padded, B * L, Kb, d, Vb, d, stream())
    dense = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    R.rocs_dca_cross_attn(Qd, Kb, Vb, offd, B, rows, L, H, dh, dh ** -0.5, dense, d, rocs.ROCS_BF16, stream(), kv_len=kv)
    assert status(R) == 0
    check_bf16(host(dense), want.reshape(rows, d), out_bf16=True, what="dense attention over what the cache gave back")
