"""GPU parity of the 4-bit history cache's calls against the float64 oracle.

Tolerances follow from what the kernels round, and nothing else:
  block tables, codes, scales, values read back: equal.
  head norms and rotation: an element is made of two products (`mag` sums their magnitudes).  fp32: the
    mean of up to 256 squares (eight fused steps and five additions in the kernel's order), the root and
    the quotient, two products, the rotation's products and sum: each at most 2^-24 relative, at most 16
    in a chain, so 16 * 2^-24 * mag; bf16 outputs round once more, 2^-8 relative to the value.
  attention: each weight is rounded to bf16 (2^-8 of it), the output is rounded to bf16 (2^-8 of it), and
    the scores carry fp32 errors: a sum of up to 128 products and the scaling, so at most
    130 * 2^-24 * scale * sum |q k|, which stays below 2^-11 for these inputs (scale * sum |q k| < 60), and
    an exponential's own 2^-21; the weights' relative error from both is below 2^-10.  With `mag` the
    weighted sum of |v|: 2^-8 (mag + |o|) + 2^-10 mag, the output's rounding taken on the rounded sum.
"""
import numpy as np
import pytest
import torch

from oracle import kv_cache as KC
from tests.gpu_util import dev_i32, host, stream
from tests.test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    from request_candidate_sharing_b200 import rocs
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    h = rocs.Rocs(0)
    yield h
    h.close()


def status(R):
    return R.rocs_get_device_status(stream())


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def dev_i64(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int64)).cuda()


# ---- block tables -----------------------------------------------------------------------------------
def run_tables(R, past, new, page, free, n_pages, table, rows):
    B = len(new)
    out = dict(table=Guarded(table.shape, torch.int32), kv=Guarded((B,), torch.int32), off=Guarded((B + 1,), torch.int32),
               slots=Guarded((rows,), torch.int64), pos=Guarded((rows,), torch.int32), used=Guarded((1,), torch.int32))
    out["table"].t.copy_(torch.from_numpy(table))
    n = R.rocs_kv_block_tables_workspace(B)
    ws = Guarded((max(n, 16),), torch.uint8)
    R.rocs_kv_block_tables(None if past is None else dev_i32(past), dev_i32(new), B, page, dev_i32(free) if len(free) else None, len(free),
                           n_pages, out["table"].t, table.shape[1], out["kv"].t, out["off"].t, out["slots"].t, out["pos"].t, rows,
                           out["used"].t, ws.t, n, stream())
    torch.cuda.synchronize()
    for k, v in list(out.items()) + [("workspace", ws)]:
        v.check(k)
    return {k: v.t.cpu().numpy() for k, v in out.items()}


def check_tables(R, past, new, page, free, n_pages, table, rows):
    got = run_tables(R, past, new, page, free, n_pages, table, rows)
    want = KC.block_tables(past, new, page, free, n_pages, table, rows)
    for k, w in zip(("table", "kv", "off", "slots", "pos"), want):
        assert np.array_equal(got[k], w), k
    assert got["used"][0] == want[5]
    code = status(R)
    assert code in {"counts": [7], "index": [5]}.get(next(iter(want[6]), None), [0]) or (len(want[6]) == 2 and code in (5, 7)), (code, want[6])


@pytest.mark.parametrize("B,page,past_top,new_top,pad", [
    (1, 16, 0, 1, 0), (1, 64, 100, 1, 3), (1, 128, 0, 40001, 7), (3, 16, 17, 33, 0), (512, 64, 1024, 1, 0), (512, 64, 0, 700, 61),
    (2048, 16, 40, 9, 1), (2049, 16, 40, 9, 0), (4096, 16, 40, 9, 1), (4097, 16, 40, 9, 0), (9001, 32, 100, 40, 5), (9000, 32, 100, 1, 5), (20000, 128, 300, 2, 4000),
])
def test_block_tables(R, B, page, past_top, new_top, pad):
    g = np.random.default_rng(B + page)
    past = g.integers(0, past_top + 1, B) if past_top else None
    new = g.integers(0 if new_top > 1 else 1, new_top + 1, B)
    p = np.zeros(B, np.int64) if past is None else past
    held, after = (p + page - 1) // page, (p + new + page - 1) // page
    need = int((after - held).sum())
    n_pages = int(held.sum()) + need + 9
    order = g.permutation(n_pages).astype(np.int32)
    table = np.full((B, max(1, int(after.max()) + int(g.integers(0, 2)))), -1, np.int32)
    k = 0
    for r in range(B):
        table[r, :held[r]] = order[k:k + held[r]]
        k += held[r]
    check_tables(R, past, new, page, order[k:], n_pages, table, int(new.sum()) + pad)


@pytest.mark.parametrize("B", [2000, 30000])
def test_block_tables_many_empty_and_some_long_requests(R, B):
    """A tile of rows that spans thousands of requests (most get nothing or one row), and one request that
    spans many tiles."""
    g = np.random.default_rng(B)
    new = (g.random(B) < 0.3).astype(np.int64)
    new[[B // 3, B - 1]] = [30011, 9000]
    past = g.integers(0, 50, B)
    page = 16
    held, after = (past + 15) // 16, (past + new + 15) // 16
    order = g.permutation(int(after.sum()) + 5).astype(np.int32)
    table = np.full((B, int(after.max())), -1, np.int32)
    k = 0
    for r in range(B):
        table[r, :held[r]] = order[k:k + held[r]]
        k += held[r]
    check_tables(R, past, new, page, order[k:], len(order), table, int(new.sum()) + 3)


@pytest.mark.parametrize("B,page,new_top,pad", [(2500, 16, 300, 9), (2100, 64, 900, 0), (2100, 16, 19000, 5)])
def test_block_tables_long_rows_of_many_requests(R, B, page, new_top, pad):
    """Rows taken request by request, among them unusable requests and bad pages; the last case has tiles whose
    part of the free list is longer than the threads keep at hand."""
    g = np.random.default_rng(B + new_top)
    new = g.integers(0, new_top + 1, B)
    past = g.integers(0, 200, B)
    held, after = (past + page - 1) // page, (past + new + page - 1) // page
    order = g.permutation(int(after.sum()) + 5).astype(np.int32)
    table = np.full((B, int(after.max())), -1, np.int32)
    k = 0
    for r in range(B):
        table[r, :held[r]] = order[k:k + held[r]]
        k += held[r]
    free = order[k:]
    check_tables(R, past, new, page, free, len(order), table, int(new.sum()) + pad)
    past[[7, 1000]] = -1, 10 ** 9                    # unusable
    table[[20, 1500], held[[20, 1500]] - 1] = -7, len(order)
    free[[3, len(free) // 2]] = -1, len(order)
    free = free[:len(free) - 400]                    # the last requests get nothing
    check_tables(R, past, new, page, free, len(order), table, int(new.sum()) - 1)


@pytest.mark.parametrize("B", [40, 5000])
def test_block_tables_bad_requests(R, B):
    """Negative and overlong lengths, a free list that runs out, bad pages in the list and in the table,
    and more rows than the outputs hold: the others keep their places."""
    g = np.random.default_rng(B)
    page, max_blocks = 16, 6
    past, new = g.integers(0, 60, B), g.integers(0, 36, B)
    past[3], new[5], new[7], past[9], past[11] = -2, -7, 200, 500, 2 ** 31 - 1
    table = np.full((B, max_blocks), -1, np.int32)
    held = np.clip((past + 15) // 16, 0, max_blocks)
    order = g.permutation(int(held.sum()) + 3 * B).astype(np.int32)
    k = 0
    for r in range(B):
        table[r, :held[r]] = order[k:k + held[r]]
        k += held[r]
    total = int(np.maximum(new, 0).sum())
    check_tables(R, past, new, page, order[k:], len(order), table, total)
    check_tables(R, past, new, page, order[k:k + B // 2], len(order), table, total)         # runs out
    check_tables(R, past, new, page, np.zeros(0, np.int32), len(order), table, total)       # nothing is free
    free = np.array(order[k:])
    free[[1, 7]] = [-5, len(order)]
    check_tables(R, past, new, page, free, len(order), table, total + 2)
    short = np.array(table)
    r = int(np.flatnonzero((past > 0) & (past % 16 != 0) & (new > 0) & (past + new < 96))[0])
    short[r, past[r] // 16] = -1
    check_tables(R, past, new, page, order[k:], len(order), short, total)
    check_tables(R, past, new, page, order[k:], len(order), table, total - 25)


def test_block_tables_slots_past_32_bits(R):
    got = run_tables(R, None, np.array([3]), 128, np.array([2 ** 31 - 2], np.int32), 2 ** 31 - 1, np.full((1, 1), -1, np.int32), 3)
    assert got["slots"].tolist() == [(2 ** 31 - 2) * 128 + j for j in range(3)] and status(R) == 0


def test_block_tables_no_rows(R):
    check_tables(R, np.array([5, 0]), np.array([0, 0]), 16, np.zeros(0, np.int32), 4, np.array([[3], [-1]], np.int32), 0)


# ---- head norms and rotation ----------------------------------------------------------------------------
@pytest.mark.parametrize("rows,Hq,Hk,d,rot,inter,io,gam", [
    (1, 1, 1, 32, 32, 0, 1, 1), (1, 8, 8, 32, 32, 1, 1, 1), (7, 8, 2, 64, 64, 0, 1, 1), (33, 3, 5, 128, 64, 0, 0, 1), (33, 3, 5, 128, 64, 1, 0, 1),
    (65, 2, 1, 256, 256, 0, 1, 1), (65, 2, 1, 256, 240, 1, 0, 1), (19, 5, 2, 80, 48, 0, 0, 1), (19, 5, 2, 80, 80, 1, 1, 1), (9, 7, 3, 16, 16, 0, 0, 1),
    (9, 2, 2, 24, 16, 0, 1, 0), (11, 4, 0, 96, 96, 0, 1, 1), (11, 0, 4, 192, 16, 1, 0, 1), (5003, 4, 2, 32, 16, 0, 1, 1), (5003, 12, 3, 64, 64, 0, 0, 0),
])
def test_qk_norm_rope(R, rows, Hq, Hk, d, rot, inter, io, gam):
    from request_candidate_sharing_b200 import rocs
    g = np.random.default_rng(rows + d)
    top, eps = 300, 1e-5
    dt = torch.bfloat16 if io else torch.float32
    width = (Hq + 2 * Hk) * d + 8                       # strided: slices of one buffer with a gap
    buf = torch.from_numpy(g.normal(size=(rows, width)).astype(np.float32)).to(dt)
    buf[0, : max(Hq, 1) * d] *= 1e-3                    # a small head, where eps counts
    x = buf.double().numpy()
    pos = g.integers(0, top, rows)
    pos[-1] = -1 if rows > 1 else pos[-1]
    pos[0] = top - 1
    cs = KC.angles(top, rot)
    gam_q, gam_k = (g.uniform(0.5, 1.5, d).astype(np.float32) for _ in range(2))
    t = buf.cuda()
    oq, ok = Guarded((rows, max(Hq, 1) * d + 8), dt, 7.0), Guarded((rows, max(Hk, 1) * d), dt, 7.0)
    desc = rocs.QkDesc(rows, Hq, Hk, d, rot, inter, top, eps, io)
    ptr = lambda a: torch.from_numpy(a).cuda() if gam else None
    gq, gk, cst, post = ptr(gam_q), ptr(gam_k), torch.from_numpy(cs).cuda(), dev_i32(pos)
    R.rocs_qk_norm_rope(desc, t if Hq else None, width, t[:, Hq * d:] if Hk else None, width, gq, gk, cst, post, oq.t if Hq else None,
                        max(Hq, 1) * d + 8, ok.t if Hk else None, max(Hk, 1) * d, stream())
    assert status(R) == 0
    oq.check("Q_out"), ok.check("K_out")
    for H, at, out, gm in ((Hq, 0, oq, gam_q), (Hk, Hq * d, ok, gam_k)):
        if not H:
            continue
        y, mag = KC.qk_norm_rope(x[:, at:at + H * d].reshape(rows, H, d), gm if gam else None, eps, cs, pos, inter)
        got = host(out.t)[:, :H * d].reshape(rows, H, d)
        live = pos >= 0
        tol = 16 * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(y) if io else 0)
        assert (np.abs(got - y) <= tol * (1 + 2.0 ** -8) + 1e-30)[live].all(), float((np.abs(got - y) / (tol + 1e-30))[live].max())
        assert (got[~live] == 7).all() and (host(out.t)[:, H * d:] == 7).all()


@pytest.mark.parametrize("inter", [0, 1])
def test_qk_norm_rope_in_place_and_bad_positions(R, inter):
    from request_candidate_sharing_b200 import rocs
    g = np.random.default_rng(7)
    rows, Hq, Hk, d = 70, 4, 2, 64
    buf = torch.from_numpy(g.normal(size=(rows, (Hq + 2 * Hk) * d)).astype(np.float32)).cuda()
    was = buf.cpu().double().numpy()
    pos = g.integers(0, 50, rows)
    pos[[4, 9]] = [50, -3]
    cs = KC.angles(50, d)
    desc = rocs.QkDesc(rows, Hq, Hk, d, d, inter, 50, 1e-6, 0)
    ld = buf.shape[1]
    k = buf[:, Hq * d:]
    post, cst = dev_i32(pos), torch.from_numpy(cs).cuda()
    R.rocs_qk_norm_rope(desc, buf, ld, k, ld, None, None, cst, post, buf, ld, k, ld, stream())
    assert status(R) == 5
    got = host(buf)
    for H, at in ((Hq, 0), (Hk, Hq * d)):
        y, mag = KC.qk_norm_rope(was[:, at:at + H * d].reshape(rows, H, d), None, 1e-6, cs, pos, inter)
        assert (np.abs(got[:, at:at + H * d].reshape(rows, H, d) - y) <= 16 * 2.0 ** -24 * mag).all()
    assert (got[[4, 9]] == was[[4, 9]]).all() and (got[:, (Hq + Hk) * d:] == was[:, (Hq + Hk) * d:]).all()


# ---- append and gather --------------------------------------------------------------------------------------
def special_rows(g, rows, H, d):
    """Rows as projections give them, with ties, zeros, tiny and huge magnitudes among them."""
    x = g.normal(size=(rows, H, d)) * np.exp(g.normal(size=(H, d)))
    x[0, 0, :32] = np.linspace(-7, 7, 32)
    if rows > 4:
        x[1, 0, :32] = np.round(g.uniform(-7, 7, 32) * 2) / 2
        x[1, 0, 0] = 7
        x[2] = 0
        x[3, 0, :32] = g.normal(size=32) * 2.0 ** -125
        x[4, 0, :32] = g.normal(size=32) * 2.0 ** 124
        x[4, -1, -1] = 3e38
    return bf16(x)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("rows,H,page", [(1, 1, 16), (5, 3, 128), (37, 8, 64), (300, 2, 32), (1000, 5, 16)])
def test_append_and_gather(R, rows, H, page, d):
    from request_candidate_sharing_b200 import rocs
    g = np.random.default_rng(rows + d)
    K, V = special_rows(g, rows, H, d), special_rows(g, rows, H, d)
    n_pages = rows // page + 3
    slots = g.permutation(n_pages * page)[:rows].astype(np.int64)
    if rows > 8:
        slots = np.sort(slots)
        slots[[6, rows - 1]] = -1
    before = g.integers(0, 256, (n_pages, H, KC.record_bytes(page, d))).astype(np.uint8)
    cache = Guarded(before.shape, torch.uint8)
    cache.t.copy_(torch.from_numpy(before))
    desc = rocs.Kv4Desc(n_pages, page, H, d)
    assert R.rocs_kv4_cache_bytes(desc) == before.size
    ldk, ldv = H * d + 8, 2 * H * d                      # strided rows
    Kd = torch.zeros(rows, ldk, dtype=torch.bfloat16, device="cuda")
    Vd = torch.zeros(rows, ldv, dtype=torch.bfloat16, device="cuda")
    Kd[:, :H * d], Vd[:, :H * d] = K.reshape(rows, -1).cuda(), V.reshape(rows, -1).cuda()
    st = dev_i64(slots)
    R.rocs_kv4_append(desc, Kd, ldk, Vd, ldv, st, rows, cache.t, stream())
    assert status(R) == 0
    cache.check("cache")
    want = KC.append(before, page, K.double().numpy(), V.double().numpy(), slots)
    assert np.array_equal(cache.t.cpu().numpy(), want)
    ko, vo = Guarded((rows, ldv), torch.bfloat16, 5.0), Guarded((rows, ldk), torch.bfloat16, 5.0)
    R.rocs_kv4_gather(desc, cache.t, st, rows, ko.t, ldv, vo.t, ldk, stream())
    assert status(R) == 0
    ko.check("K"), vo.check("V")
    live = slots >= 0
    for out, x in ((ko, K), (vo, V)):
        codes, s = KC.quantize(x.double().numpy())
        got = host(out.t)
        assert np.array_equal(got[live][:, :H * d], KC.dequantize(codes, s).reshape(rows, -1)[live])
        assert (got[~live] == 5).all() and (got[:, H * d:] == 5).all()


def test_append_bad_slots_and_values(R):
    from request_candidate_sharing_b200 import rocs
    g = np.random.default_rng(5)
    H, d, page, n_pages = 2, 64, 16, 2
    K, V = special_rows(g, 4, H, d), special_rows(g, 4, H, d)
    desc = rocs.Kv4Desc(n_pages, page, H, d)
    cache = Guarded((n_pages, H, KC.record_bytes(page, d)), torch.uint8)
    cache.t.zero_()
    slots = np.array([32, 3, -2, 2 ** 40])
    R.rocs_kv4_append(desc, K.cuda(), H * d, V.cuda(), H * d, dev_i64(slots), 4, cache.t, stream())
    assert status(R) == 5
    cache.check("cache")
    zero = np.zeros(cache.t.shape, np.uint8)
    assert np.array_equal(cache.t.cpu().numpy(), KC.append(zero, page, K.double().numpy(), V.double().numpy(), slots))
    out = torch.full((4, H * d), 5.0, dtype=torch.bfloat16, device="cuda")
    R.rocs_kv4_gather(desc, cache.t, dev_i64(slots), 4, out, H * d, torch.empty_like(out), H * d, stream())
    assert status(R) == 5 and (host(out)[[0, 2, 3]] == 5).all()
    for bad in (float("nan"), float("inf"), -float("inf")):
        K[1, 0, 40], V[2, 1, 3] = bad, bad
        R.rocs_kv4_append(desc, K.cuda(), H * d, V.cuda(), H * d, dev_i64([0, 1, 2, 3]), 4, cache.t, stream())
        assert status(R) == 8
        got = cache.t.cpu().numpy()
        assert np.array_equal(got, KC.append(got, page, K.double().numpy(), V.double().numpy(), [0, 1, 2, 3]))


# ---- attention -------------------------------------------------------------------------------------------------
class Cached:
    """Random requests over a cache: pages anywhere, garbage (NaN scales among it) past each end."""

    def __init__(self, seed, counts, lens, H_kv, share, d, page, pad_rows=0, spare_blocks=1):
        g = np.random.default_rng(seed)
        self.counts, self.lens = np.asarray(counts), np.asarray(lens)
        self.H, self.share, self.d, self.page = H_kv, share, d, page
        self.rows = int(self.counts.sum()) + pad_rows
        self.offsets = np.concatenate([[0], np.cumsum(self.counts)])
        held = (self.lens + page - 1) // page
        self.n_pages = int(held.sum()) + 3
        order = g.permutation(self.n_pages)
        self.max_blocks = max(1, int(held.max()) + spare_blocks)
        self.table = np.full((len(counts), self.max_blocks), -1, np.int32)
        cache = g.integers(0, 256, (self.n_pages, H_kv, KC.record_bytes(page, d))).astype(np.uint8)
        for kv in (0, 1):                                # every scale NaN until written
            half = KC.record_bytes(page, d) // 2
            cache[:, :, kv * half + page * d // 2:(kv + 1) * half] = 0xFF
        k, slots = 0, []
        for r in range(len(counts)):
            self.table[r, :held[r]] = order[k:k + held[r]]
            k += held[r]
            t = np.arange(self.lens[r])
            slots.append(self.table[r, t // page].astype(np.int64) * page + t % page)
        slots = np.concatenate(slots) if len(slots) else np.zeros(0, np.int64)
        rnd = lambda *s: bf16(g.normal(size=s)).double().numpy()
        self.cache = KC.append(cache, page, rnd(len(slots), H_kv, d), rnd(len(slots), H_kv, d), slots)
        self.K, self.V = KC.values(self.cache, page, d)
        self.Q = rnd(self.rows, H_kv * share, d)

    def want(self, scale, causal):
        return KC.attention(self.Q, self.H, self.K, self.V, self.table, self.lens, self.offsets, self.page, scale, causal)

    def run(self, R, scale, causal, ld_extra=0, kv_len=None, offsets=None, table=None, Q=None):
        from request_candidate_sharing_b200 import rocs
        Hq = self.H * self.share
        ld = Hq * self.d + ld_extra
        desc = rocs.Kv4Desc(self.n_pages, self.page, self.H, self.d)
        B = len(self.counts)
        Qd = torch.full((self.rows, ld), float("nan"), dtype=torch.bfloat16)
        Qd[:, :Hq * self.d] = bf16(self.Q if Q is None else Q).reshape(self.rows, -1)
        out = Guarded((self.rows, ld), torch.bfloat16, 9.0)
        n = R.rocs_dca_cross_attn_kv4_workspace(desc, Hq, B, self.rows, self.max_blocks)
        ws = Guarded((max(n, 16),), torch.uint8)
        ws.t.fill_(255)
        R.rocs_dca_cross_attn_kv4(desc, Qd.cuda(), ld, Hq, torch.from_numpy(self.cache).cuda(), dev_i32(self.table if table is None else table),
                                  self.max_blocks, dev_i32(self.lens if kv_len is None else kv_len),
                                  dev_i32(self.offsets if offsets is None else offsets), B, self.rows, scale, causal, out.t, ld, ws.t, n, stream())
        torch.cuda.synchronize()
        out.check("O"), ws.check("workspace")
        got = host(out.t)
        assert (got[:, Hq * self.d:] == 9).all()
        return got[:, :Hq * self.d].reshape(self.rows, Hq, self.d)


def close(got, want, mag):
    tol = 2.0 ** -8 * (mag + np.abs(want)) * (1 + 2.0 ** -8) + 2.0 ** -10 * mag
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


ONE = [([1], [1]), ([1], [63]), ([1, 1, 1], [64, 0, 65]), ([1] * 40, list(range(0, 400, 10)))]
FEW = [([3, 0, 5, 2], [100, 50, 0, 129]), ([8, 9, 1], [16, 17, 300]), ([16, 20, 13], [64, 128, 191])]
MANY = [([40, 0, 33, 200], [70, 5, 300, 257]), ([128, 129, 1], [512, 1, 90])]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("counts,lens", ONE + FEW + MANY)
def test_attention(R, counts, lens, d, page):
    c = Cached(1, counts, lens, 2, 1, d, page)
    close(c.run(R, d ** -0.5, 0, ld_extra=8), *c.want(d ** -0.5, 0))
    assert status(R) == 0


@pytest.mark.parametrize("H,share", [(1, 1), (3, 1), (1, 2), (2, 3), (1, 8), (2, 8), (1, 16), (1, 37)])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("counts,lens", [ONE[3], FEW[0], MANY[1]])
def test_attention_shared_heads(R, counts, lens, d, H, share):
    c = Cached(2, counts, lens, H, share, d, 64)
    close(c.run(R, d ** -0.5, 0), *c.want(d ** -0.5, 0))
    assert status(R) == 0


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("d,share", [(32, 1), (64, 2), (128, 4)])
@pytest.mark.parametrize("counts,lens", [([1, 1], [1, 77]), ([5, 3, 64, 0], [5, 2, 64, 30]), ([7, 130, 70], [200, 130, 333]), ([300], [290])])
def test_attention_causal(R, counts, lens, d, share, page):
    """Rows see up to themselves; where a request has more rows than keys its first rows see nothing."""
    c = Cached(3, counts, lens, 2, share, d, page)
    close(c.run(R, d ** -0.5, 1), *c.want(d ** -0.5, 1))
    assert status(R) == 0


@pytest.mark.parametrize("d,share,counts,lens", [(32, 1, [1], [20000]), (64, 4, [1, 1], [9000, 16385]), (128, 1, [2], [12345]), (64, 1, [40], [8000])])
def test_attention_long_histories_are_split(R, d, share, counts, lens):
    c = Cached(4, counts, lens, 1, share, d, 64)
    close(c.run(R, d ** -0.5, 0), *c.want(d ** -0.5, 0))
    close(c.run(R, d ** -0.5, 1), *c.want(d ** -0.5, 1))
    assert status(R) == 0


@pytest.mark.parametrize("counts,lens", [([1] * 5, [30, 0, 64, 65, 1]), ([60, 70], [100, 200])])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5])
def test_attention_scales(R, counts, lens, scale):
    """A scale of 0 weighs all keys alike; a negative one turns the order round; a large one makes rows
    of one weight."""
    c = Cached(5, counts, lens, 2, 1, 32, 32)
    close(c.run(R, scale, 0), *c.want(scale, 0))


@pytest.mark.parametrize("counts", [[1, 1, 1], [50, 60, 70]])
def test_attention_padded_rows_and_foreign_rows_stay(R, counts):
    c = Cached(6, counts, [40, 0, 100], 2, 1, 64, 16, pad_rows=5)
    got = c.run(R, 0.125, 0)
    want, mag = c.want(0.125, 0)
    n = int(c.offsets[-1])
    close(got[:n], want[:n], mag[:n])
    assert (got[n:] == 9).all() and status(R) == 0


@pytest.mark.parametrize("counts", [[1, 1, 1, 1], [40, 50, 30, 60]])
def test_attention_non_finite_queries_touch_their_rows_only(R, counts):
    c = Cached(7, counts, [90, 64, 300, 17], 2, 2, 64, 64)
    Q = np.array(c.Q)
    row = int(c.offsets[1])
    Q[row, 1, 5], Q[row, 2, :] = np.nan, np.inf
    got = c.run(R, 0.125, 0, Q=Q)
    want, mag = c.want(0.125, 0)
    keep = np.ones(got.shape[:2], bool)
    keep[row, 1:3] = False
    close(got[keep], want[keep], mag[keep])
    assert np.isnan(got[row, 1:3]).all()


@pytest.mark.parametrize("counts", [[1, 2, 1, 3], [40, 50, 30, 60]])
def test_attention_bad_lengths_and_offsets(R, counts):
    c = Cached(8, counts, [90, 64, 300, 17], 2, 1, 64, 64)
    want, mag = c.want(0.125, 0)
    o = c.offsets
    for bad in (-1, c.max_blocks * 64 + 1, 2 ** 31 - 1):
        lens = np.array(c.lens)
        lens[1] = bad
        got = c.run(R, 0.125, 0, kv_len=lens)
        keep = np.r_[0:o[1], o[2]:o[4]]
        close(got[keep], want[keep], mag[keep])
        assert (got[o[1]:o[2]] == 9).all() and status(R) == 7
    off = np.array(o)
    off[4] = c.rows + 1                                   # the last request reaches past the rows
    got = c.run(R, 0.125, 0, offsets=off)
    close(got[:o[3]], want[:o[3]], mag[:o[3]])
    assert (got[o[3]:] == 9).all() and status(R) == 5
    n = c.rows
    for off in ([-5, 3, 2, 2 ** 31 - 1, 1], [4, 3, 2, 1, 0], [0, n, 0, n, 0], [0, n, n - 1, n, n]):
        c.run(R, 0.125, 0, offsets=np.array(off))
        assert status(R) == 5


@pytest.mark.parametrize("q", [1, 40])
def test_attention_offsets_that_go_back_and_forth(R, q):
    """Thousands of requests that all claim every row: refused on the device, within the workspace."""
    c = Cached(14, [q] * 300, [40] * 300, 2, 1, 32, 16)
    off = np.where(np.arange(301) % 2 == 0, 0, c.rows)
    got = c.run(R, 0.2, 0, offsets=off)
    assert status(R) == 5 and ((got == 9).all() or not np.isnan(got).any())


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("counts", [[1, 1], [70, 9]])
def test_attention_missing_pages_are_left_out(R, counts, page):
    """A page that does not exist: its keys are left out and the status says so."""
    c = Cached(9, counts, [300, 200], 2, 1, 32, page)
    table = np.array(c.table)
    table[0, 1] = c.n_pages
    got = c.run(R, 0.2, 0, table=table)
    assert status(R) == 5
    want, mag = c.want(0.2, 0)
    n = c.counts[0]
    close(got[n:], want[n:], mag[n:])
    keys = np.r_[0:page, min(2 * page, 300):300]
    for h in range(2):
        k, v = (x[c.table[0, :-(-300 // page)], h].reshape(-1, 32)[keys] for x in (c.K, c.V))
        s = c.Q[:n, h] @ k.T * 0.2
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        close(got[:n, h], w @ v, w @ np.abs(v))


@pytest.mark.parametrize("q,d,causal", [(1, 32, 0), (1, 64, 1), (34, 32, 0), (34, 32, 1)])
def test_attention_more_requests_than_are_listed(R, q, d, causal):
    """Past 8192 requests the blocks find their tiles themselves, for few rows and for many."""
    B = 8200
    g = np.random.default_rng(q)
    counts = np.full(B, q)
    counts[g.integers(0, B, 200)] = 0
    counts[77] += 150
    lens = g.integers(0, 60 if q == 1 else 20, B)
    c = Cached(15, counts, lens, 1, 1, d, 16)
    bad = np.array(c.lens)
    bad[[5, 8000]] = [-1, c.max_blocks * 16 + 1]
    got = c.run(R, d ** -0.5, causal, kv_len=bad)
    assert status(R) == 7
    want, mag = c.want(d ** -0.5, causal)
    keep = np.ones(c.rows, bool)
    for r in (5, 8000):
        keep[c.offsets[r]:c.offsets[r + 1]] = False
    close(got[keep], want[keep], mag[keep])
    assert (got[~keep] == 9).all()


@pytest.mark.parametrize("d,q", [(32, 40), (64, 150), (128, 65)])
def test_attention_runs_of_empty_and_tiny_histories(R, d, q):
    """Hundreds of histories of no, one or a few blocks in a row: the tiles of one block of threads follow each other."""
    B = 1500
    g = np.random.default_rng(d)
    lens = g.choice([0, 0, 0, 0, 1, 63, 64, 65, 130], B)
    lens[200:900] = 0
    lens[1200:] = g.integers(1, 3, 300)
    c = Cached(19, g.integers(q - 8, q + 8, B), lens, 1, 1, d, 16)
    for causal in (0, 1):
        got = c.run(R, d ** -0.5, causal)
        assert status(R) == 0
        close(got, *c.want(d ** -0.5, causal))


@pytest.mark.parametrize("counts,lens,d,share,page", [
    ([1, 1, 1, 1, 1], [30000, 1, 0, 9000, 4097], 64, 2, 64), ([1] * 700, [(37 * i) % 900 for i in range(700)], 32, 1, 64),
    ([100, 3, 260, 0, 31], [9000, 4000, 700, 50, 1], 128, 1, 128), ([200, 500, 40, 129], [64, 1000, 333, 2049], 32, 2, 16),
])
def test_attention_replayed_from_a_graph(R, counts, lens, d, share, page):
    """The listed, split and joined forms, replayed with other queries and lengths of the same buffers."""
    from request_candidate_sharing_b200 import rocs
    c = Cached(16, counts, lens, 2, share, d, page)
    Hq, B = 2 * share, len(counts)
    desc, ld = rocs.Kv4Desc(c.n_pages, page, 2, d), 2 * share * d
    n = R.rocs_dca_cross_attn_kv4_workspace(desc, Hq, B, c.rows, c.max_blocks)
    assert n > 0
    t = dict(q=bf16(c.Q).reshape(c.rows, -1).cuda(), cache=torch.from_numpy(c.cache).cuda(), table=dev_i32(c.table), kv=dev_i32(c.lens),
             off=dev_i32(c.offsets), out=torch.zeros(c.rows, ld, dtype=torch.bfloat16, device="cuda"),
             ws=torch.full((n,), 255, dtype=torch.uint8, device="cuda"))

    def call(s):
        R.rocs_dca_cross_attn_kv4(desc, t["q"], ld, Hq, t["cache"], t["table"], c.max_blocks, t["kv"], t["off"], B, c.rows, d ** -0.5, 1, t["out"], ld,
                                  t["ws"], n, s.cuda_stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(side)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call(side)
            call(side)                      # twice in one graph, with one workspace: in order
        rng = np.random.default_rng(1)
        for step in range(3):
            if step:
                c.lens = np.array([rng.integers(0, x + 1) for x in lens])
                c.Q = bf16(rng.normal(size=c.Q.shape)).double().numpy()
                t["kv"].copy_(dev_i32(c.lens))
                t["q"].copy_(bf16(c.Q).reshape(c.rows, -1).cuda())
            t["out"].fill_(9.0)
            g.replay()
            side.synchronize()
            assert R.rocs_get_device_status(side.cuda_stream) == 0
            close(host(t["out"]).reshape(c.rows, Hq, d), *c.want(d ** -0.5, 1))
    del g


@pytest.mark.parametrize("counts,lens", [([1], [60000]), ([3, 1], [9000, 20000]), ([200], [5000])])
def test_attention_same_bits_every_time(R, counts, lens):
    """Lists and partial results are laid out by atomics; the results do not depend on their order."""
    c = Cached(17, counts, lens, 4, 1, 64, 64)
    first = c.run(R, 0.125, 0)
    for _ in range(5):
        assert np.array_equal(c.run(R, 0.125, 0), first)


def test_attention_no_rows(R):
    from request_candidate_sharing_b200 import rocs
    d = rocs.Kv4Desc(3, 16, 1, 32)
    i = dev_i32([0, 0])
    R.rocs_dca_cross_attn_kv4(d, None, 32, 1, torch.zeros(3 * 576, dtype=torch.uint8, device="cuda"), i, 1, i, i, 1, 0, 1.0, 0, None, 32, None, 0,
                              stream())
    assert status(R) == 0


@pytest.mark.parametrize("d,page", [(32, 16), (64, 64), (128, 128)])
def test_attention_many_rows_cache_offsets_past_32_bits(R, d, page):
    """150 candidates against the last two pages of a cache of 5 GB."""
    from request_candidate_sharing_b200 import rocs
    H = 8
    rec = KC.record_bytes(page, d)
    n_pages = 5 * 2 ** 30 // (H * rec)
    cache = torch.empty(n_pages, H, rec, dtype=torch.uint8, device="cuda")
    length = 2 * page - 3
    c = Cached(20, [150], [length], H, 1, d, page)
    cache[-2:].copy_(torch.from_numpy(c.cache[c.table[0, :2]]))
    desc = rocs.Kv4Desc(n_pages, page, H, d)
    out = torch.zeros(150, H * d, dtype=torch.bfloat16, device="cuda")
    q, table = bf16(c.Q).reshape(150, -1).cuda(), dev_i32([[n_pages - 2, n_pages - 1]])
    n = R.rocs_dca_cross_attn_kv4_workspace(desc, H, 1, 150, 2)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    R.rocs_dca_cross_attn_kv4(desc, q, H * d, H, cache, table, 2, dev_i32([length]), dev_i32([0, 150]), 1, 150, 0.1, 1, out, H * d, ws, n, stream())
    assert status(R) == 0
    close(host(out).reshape(150, H, d), *c.want(0.1, 1))


def test_attention_cache_offsets_past_32_bits(R):
    """The last page of a cache of 5 GB."""
    from request_candidate_sharing_b200 import rocs
    page, H, d = 128, 8, 128
    rec = KC.record_bytes(page, d)
    n_pages = 5 * 2 ** 30 // (H * rec)
    cache = torch.empty(n_pages, H, rec, dtype=torch.uint8, device="cuda")
    c = Cached(10, [2], [128], H, 1, d, page)
    cache[-1].copy_(torch.from_numpy(c.cache[c.table[0, 0]]))
    desc = rocs.Kv4Desc(n_pages, page, H, d)
    out = torch.zeros(2, H * d, dtype=torch.bfloat16, device="cuda")
    q, table, ln, off = bf16(c.Q).reshape(2, -1).cuda(), dev_i32([[n_pages - 1]]), dev_i32([128]), dev_i32([0, 2])
    n = R.rocs_dca_cross_attn_kv4_workspace(desc, H, 1, 2, 1)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    R.rocs_dca_cross_attn_kv4(desc, q, H * d, H, cache, table, 1, ln, off, 1, 2, 0.1, 0, out, H * d, ws, n, stream())
    close(host(out).reshape(2, H, d), *c.want(0.1, 0))
    back = torch.zeros(2, 128, H * d, dtype=torch.bfloat16, device="cuda")
    slots = dev_i64(np.arange(128) + (n_pages - 1) * page)
    R.rocs_kv4_gather(desc, cache, slots, 128, back[0], H * d, back[1], H * d, stream())
    for x, want in zip(back, (c.K, c.V)):
        assert np.array_equal(host(x).reshape(128, H, d), want[c.table[0, 0]].transpose(1, 0, 2))
    R.rocs_kv4_append(desc, back[0], H * d, back[1], H * d, slots, 128, cache, stream())
    again = torch.zeros_like(back)
    R.rocs_kv4_gather(desc, cache, slots, 128, again[0], H * d, again[1], H * d, stream())
    for x, y in zip(back, again):      # stored again: a group whose largest code was 6 takes a smaller scale
        want = KC.dequantize(*KC.quantize(host(x).reshape(128, H, d))).reshape(128, -1)
        assert np.array_equal(host(y), want)
    assert status(R) == 0


# ---- the calls together -----------------------------------------------------------------------------------------
class Step:
    """Serving steps as a program makes them: its buffers, and one step's four calls."""

    def __init__(self, R, B, H, share, d, page, max_blocks, n_pages, max_rows):
        from request_candidate_sharing_b200 import rocs
        self.R, self.B, self.H, self.share, self.d, self.page, self.max_blocks, self.rows = R, B, H, share, d, page, max_blocks, max_rows
        self.rocs = rocs
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        self.past, self.new, self.kv, self.off, self.used = i32(B), i32(B), i32(B), i32(B + 1), i32(1)
        self.free = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).int().cuda()
        self.table = torch.full((B, max_blocks), -1, dtype=torch.int32, device="cuda")
        self.slots = torch.zeros(max_rows, dtype=torch.int64, device="cuda")
        self.pos = i32(max_rows)
        self.n_pages = n_pages
        self.desc = rocs.Kv4Desc(n_pages, page, H, d)
        self.cache = torch.full((R.rocs_kv4_cache_bytes(self.desc),), 255, dtype=torch.uint8, device="cuda")
        self.width = (H * share + 2 * H) * d
        self.qkv = torch.zeros(max_rows, self.width, dtype=torch.bfloat16, device="cuda")
        self.gamma = torch.linspace(0.5, 1.5, d, device="cuda")
        self.cs = torch.from_numpy(KC.angles(max_blocks * page, d)).cuda()
        self.out = torch.full((max_rows, H * share * d), 9.0, dtype=torch.bfloat16, device="cuda")
        n = R.rocs_dca_cross_attn_kv4_workspace(self.desc, H * share, B, max_rows, max_blocks)
        self.ws, self.ws_n = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), n

    def calls(self):
        R, H, d, Hq, s = self.R, self.H, self.d, self.H * self.share, torch.cuda.current_stream().cuda_stream
        k, v = self.qkv[:, Hq * d:], self.qkv[:, (Hq + H) * d:]
        R.rocs_kv_block_tables(self.past, self.new, self.B, self.page, self.free, self.free.numel(), self.n_pages, self.table, self.max_blocks,
                               self.kv, self.off, self.slots, self.pos, self.rows, self.used, None, 0, s)
        qd = self.rocs.QkDesc(self.rows, Hq, H, d, d, 0, self.max_blocks * self.page, 1e-6, 1)
        R.rocs_qk_norm_rope(qd, self.qkv, self.width, k, self.width, self.gamma, self.gamma, self.cs, self.pos, self.qkv, self.width, k, self.width, s)
        R.rocs_kv4_append(self.desc, k, self.width, v, self.width, self.slots, self.rows, self.cache, s)
        R.rocs_dca_cross_attn_kv4(self.desc, self.qkv, self.width, Hq, self.cache, self.table, self.max_blocks, self.kv, self.off, self.B, self.rows,
                                  d ** -0.5, 1, self.out, Hq * d, self.ws, self.ws_n, s)


def reference_step(hist, new, qkv, off, H, share, d, page, gamma, cs):
    """What a step's outputs should be, with the histories kept as plain lists: normed and rotated as
    bf16, stored as 4-bit values."""
    Hq = H * share
    rows = int(off[-1])
    x = qkv[:rows].reshape(rows, Hq + 2 * H, d)
    out, mag = np.zeros((rows, Hq, d)), np.zeros((rows, Hq, d))
    for r in range(len(new)):
        a, b = int(off[r]), int(off[r + 1])
        hist[r].append(x[a:b])
    for r in range(len(new)):
        a, b = int(off[r]), int(off[r + 1])
        if a == b:
            continue
        allx = np.concatenate(hist[r])
        kv = []
        for y in (allx[:, Hq:Hq + H], allx[:, Hq + H:]):
            codes, s = KC.quantize(y)
            kv.append(KC.dequantize(codes, s))
        n = len(allx)
        K, V = (y.transpose(1, 0, 2)[None] for y in kv)      # one page that holds all
        out[a:b], mag[a:b] = KC.attention(x[a:b, :Hq], H, K, V, np.zeros((1, 1), int), [n], [0, b - a], n, d ** -0.5, 1)
    return out, mag


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("B,H,share,d,page", [(4, 2, 2, 64, 16), (3, 2, 1, 32, 64)])
def test_serving_steps(R, B, H, share, d, page, graph):
    """Histories come in, then single events and bursts; every step runs all four calls, eagerly on a
    stream of its own or replayed from one captured graph with padded rows."""
    g = np.random.default_rng(B)
    rows = 96
    st = Step(R, B, H, share, d, page, 8, 60, rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    news = [g.integers(10, 25, B), np.ones(B, int), np.array([1, 0, 17] + [3] * (B - 3)), np.ones(B, int)]
    cg = None
    hist = [[] for _ in range(B)]
    for step, new in enumerate(news):
        x = bf16(g.normal(size=(rows, st.width)))
        with torch.cuda.stream(side):
            st.new.copy_(dev_i32(new))
            st.qkv.copy_(x.cuda())
            if graph and cg is None:
                st.new.zero_()
                st.calls()                                # warm-up: no new events
                side.synchronize()
                cg = torch.cuda.CUDAGraph()
                with torch.cuda.graph(cg, stream=side):
                    st.calls()
                st.new.copy_(dev_i32(new))
                st.qkv.copy_(x.cuda())
            if graph:
                cg.replay()
            else:
                st.calls()
            side.synchronize()
            assert R.rocs_get_device_status(side.cuda_stream) == 0
            off = st.off.cpu().numpy()
            n = int(off[-1])
            assert n == new.sum() and (st.kv.cpu().numpy() == st.past.cpu().numpy() + new).all()
            qkv = host(st.qkv)
            # the normed rows are checked by their own test; here their bf16 values feed the reference
            want, mag = reference_step(hist, new, qkv, off, H, share, d, page, None, None)
            got = host(st.out).reshape(rows, H * share, d)
            close(got[:n], want, mag)
            assert (got[n:] == 9).all()
            st.out.fill_(9.0)
            # the next step: what is cached, and the pages left
            st.past.copy_(st.kv)
            used = int(st.used.item())
            st.free.copy_(torch.cat([st.free[used:], st.free[:used]]))
    del cg


def test_calls_refuse_another_current_device_or_small_workspace(R):
    from request_candidate_sharing_b200 import rocs
    c = Cached(11, [1], [20000], 1, 1, 32, 64)
    d = rocs.Kv4Desc(c.n_pages, 64, 1, 32)
    n = R.rocs_dca_cross_attn_kv4_workspace(d, 1, 1, 1, c.max_blocks)
    assert n > 0
    t = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    for ws, size in ((None, n), (t, n - 1), (t.data_ptr() + 16, n)):
        with pytest.raises(rocs.RocsError) as e:
            R.rocs_dca_cross_attn_kv4(d, t, 32, 1, t, t, c.max_blocks, t, t, 1, 1, 1.0, 0, t, 32, ws, size, stream())
        assert e.value.status == rocs.ROCS_ERR_WORKSPACE


@pytest.mark.parametrize("at", [0, 16, 4096 + 512, 9216 + 256, 20480, 24576, 28672])
def test_attention_refuses_an_output_over_its_inputs(R, at):
    """Q at 0, the cache at 9216, then the table, the lengths and the offsets."""
    from request_candidate_sharing_b200 import rocs
    d = rocs.Kv4Desc(16, 16, 1, 32)            # 9216 bytes
    t = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    a = t.data_ptr()
    n = R.rocs_dca_cross_attn_kv4_workspace(d, 8, 1, 10, 1)
    assert a % 256 == 0 and n <= 32768
    with pytest.raises(rocs.RocsError) as e:
        R.rocs_dca_cross_attn_kv4(d, a, 256, 8, a + 9216, a + 20480, 1, a + 24576, a + 28672, 1, 10, 1.0, 0, a + at, 256, a + 32768, n, stream())
    assert e.value.status == rocs.ROCS_ERR_INVALID_ARG and "overlaps" in str(e.value)


def test_attention_output_beside_the_queries_in_one_buffer(R):
    c = Cached(18, [3, 0, 50], [40, 10, 33], 2, 2, 32, 16)
    from request_candidate_sharing_b200 import rocs
    desc = rocs.Kv4Desc(c.n_pages, 16, 2, 32)
    buf = torch.zeros(c.rows, 256, dtype=torch.bfloat16, device="cuda")
    buf[:, :128] = bf16(c.Q).reshape(c.rows, -1).cuda()
    n = R.rocs_dca_cross_attn_kv4_workspace(desc, 4, 3, c.rows, c.max_blocks)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    R.rocs_dca_cross_attn_kv4(desc, buf, 256, 4, torch.from_numpy(c.cache).cuda(), dev_i32(c.table), c.max_blocks, dev_i32(c.lens),
                              dev_i32(c.offsets), 3, c.rows, 0.2, 0, buf[:, 128:], 256, ws, n, stream())
    assert status(R) == 0
    close(host(buf[:, 128:]).reshape(c.rows, 4, 32), *c.want(0.2, 0))


def test_calls_refuse_when_another_device_is_current(R):
    """A handle of another device (only its number is looked at before the refusal)."""
    import ctypes
    from request_candidate_sharing_b200 import rocs
    fake = ctypes.create_string_buffer(256)
    ctypes.memmove(fake, ctypes.byref(ctypes.c_int32(3)), 4)
    h = ctypes.cast(fake, ctypes.c_void_p)
    t = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    a = t.data_ptr()
    d, q = rocs.Kv4Desc(3, 16, 1, 32), rocs.QkDesc(1, 1, 1, 32, 32, 0, 8, 1e-6, 1)
    calls = [lambda: rocs._lib_tab(h, a, a + 256, 1, 16, a + 512, 1, 3, a + 1024, 1, a + 1280, a + 1536, a + 2048, a + 2304, 1, a + 2560, None, 0, None),
             lambda: rocs._lib_qk(h, ctypes.byref(q), a, 32, a + 256, 32, None, None, a + 512, a + 2048, a + 4096, 32, a + 4352, 32, None),
             lambda: rocs._lib_kv4_app(h, ctypes.byref(d), a, 32, a + 256, 32, a + 512, 1, a + 4096, None),
             lambda: rocs._lib_kv4_get(h, ctypes.byref(d), a + 4096, a + 512, 1, a, 32, a + 256, 32, None),
             lambda: rocs._lib_attn4(h, ctypes.byref(d), a, 32, 1, a + 4096, a + 512, 1, a + 768, a + 1024, 1, 1, 1.0, 0, a + 1280, 32, None, 0, None)]
    for call in calls:
        assert call() == rocs.ROCS_ERR_INVALID_ARG and "is current" in rocs.rocs_last_error()


def test_two_streams_at_once(R):
    """Two calls with their own workspaces on two streams give what they give alone."""
    a, b = Cached(12, [1, 1], [9000, 3000], 2, 1, 64, 64), Cached(13, [70], [5000], 2, 1, 64, 16)
    wa, wb = a.want(0.125, 0), b.want(0.125, 0)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    from request_candidate_sharing_b200 import rocs
    jobs = []
    for c, s in ((a, s1), (b, s2)):
        desc = rocs.Kv4Desc(c.n_pages, c.page, c.H, c.d)
        B, ld = len(c.counts), c.H * c.d
        n = R.rocs_dca_cross_attn_kv4_workspace(desc, c.H, B, c.rows, c.max_blocks)
        t = dict(q=bf16(c.Q).reshape(c.rows, -1).cuda(), cache=torch.from_numpy(c.cache).cuda(), table=dev_i32(c.table), kv=dev_i32(c.lens),
                 off=dev_i32(c.offsets), out=torch.zeros(c.rows, ld, dtype=torch.bfloat16, device="cuda"),
                 ws=torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"))
        jobs.append((c, s, desc, B, ld, n, t))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, desc, B, ld, n, t in jobs:
            R.rocs_dca_cross_attn_kv4(desc, t["q"], ld, c.H, t["cache"], t["table"], c.max_blocks, t["kv"], t["off"], B, c.rows, 0.125, 0, t["out"], ld,
                                      t["ws"], n, s.cuda_stream)
    torch.cuda.synchronize()
    for (c, _, _, _, _, _, t), w in zip(jobs, (wa, wb)):
        close(host(t["out"]).reshape(c.rows, c.H, c.d), *w)
    assert status(R) == 0
