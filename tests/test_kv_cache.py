"""The 4-bit history cache without a GPU: what the oracle's definitions say, pinned by hand, by
brute force and against torch, and the entry points' refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv_cache as KC
from oracle import rocs_oracle as O


# ---- the oracle -----------------------------------------------------------------------------------
def test_block_tables_by_hand():
    # page of 4: request 0 holds 3 tokens in page 9 and gets 3 (one fresh page), request 1 holds 4 in
    # page 5 and gets 1 (a full page: fresh), request 2 gets none, request 3 starts with 5
    table = np.array([[9, -1], [5, -1], [-1, -1], [-1, -1]], np.int32)
    t, kv, off, slots, pos, used, st = KC.block_tables([3, 4, 0, 0], [3, 1, 0, 5], 4, [7, 2, 0, 1, 3], 10, table, 11)
    assert t.tolist() == [[9, 7], [5, 2], [-1, -1], [0, 1]]
    assert kv.tolist() == [6, 5, 0, 5] and off.tolist() == [0, 3, 4, 4, 9] and used == 4 and st == set()
    assert slots.tolist() == [39, 28, 29, 8, 0, 1, 2, 3, 4, -1, -1]
    assert pos.tolist() == [3, 4, 5, 4, 0, 1, 2, 3, 4, -1, -1]


def test_block_tables_out_of_pages_and_bad_lengths():
    table = np.full((4, 2), -1, np.int32)
    t, kv, off, slots, pos, used, st = KC.block_tables([0, -1, 0, 0], [4, 2, 9, 5], 4, [3, 1], 10, table, 20)
    # request 1 and 2 have unusable lengths, request 3 wants two pages and one is left
    assert kv.tolist() == [4, 0, 0, 0] and used == 1 and st == {"counts"} and off.tolist() == [0, 4, 6, 15, 20]
    assert slots.tolist()[:4] == [12, 13, 14, 15] and (slots[4:] == -1).all() and t[0, 0] == 3 and (t[1:] == -1).all()


def test_scale_is_the_smallest_four_bit_number_that_fits():
    g = np.random.default_rng(0)
    four = np.sort(np.concatenate([np.arange(8, 16) * 2.0 ** e for e in range(-60, 8)]))
    for top in np.concatenate([np.abs(g.normal(size=300)), 7 * four[400:440], 7 * four[400:440] * (1 + 2.0 ** -8)]):
        s = float(KC.scale_of(top))
        assert s == four[np.searchsorted(four, top / 7)]
    assert KC.scale_of(0.0) == 2.0 ** -120 and KC.scale_of(1e38) == 2.0 ** 120


def test_every_stored_value_is_a_bf16_number():
    mant = np.array([m * 2.0 ** e for m in range(8, 16) for e in (-123, -10, 0, 5, 117)])
    v = np.concatenate([mant * q for q in range(-7, 8)]).astype(np.float32)
    assert (torch.from_numpy(v).to(torch.bfloat16).float().numpy() == v).all()
    # and so is the constant of the kernels' dequantisation, (128 + n) s - 136 s
    c = (mant * 136).astype(np.float32)
    assert (torch.from_numpy(c).to(torch.bfloat16).float().numpy() == c).all()


def test_quantize_is_nearest_with_ties_away_from_zero():
    g = np.random.default_rng(1)
    x = torch.from_numpy(g.normal(size=(64, 64)).astype(np.float32)).to(torch.bfloat16).double().numpy()
    x[0, :3] = [7.0, 2.5, -2.5]     # scale 1 in this group: ties
    x[0, 3:32] = 0.25
    codes, s = KC.quantize(x)
    back = KC.dequantize(codes, s)
    assert codes[0, :3].tolist() == [15, 11, 5]
    step = np.repeat(s, 32, -1)
    assert (np.abs(back - x) <= step / 2).all() and codes.min() >= 1 and codes.max() <= 15
    for i in range(x.shape[0]):      # no other code is nearer
        for c in range(1, 16):
            assert (np.abs((c - 8) * step[i] - x[i]) >= np.abs(back[i] - x[i]) - 1e-300).all()


def test_record_layout_by_hand():
    page, d, H = 16, 32, 2
    cache = np.zeros((3, H, KC.record_bytes(page, d)), np.uint8)
    K, V = np.zeros((1, H, d)), np.zeros((1, H, d))
    K[0, 1, :4] = [7, -3, 1, 0]      # scale 1
    V[0, 1, 31] = 14                 # scale 2
    c = KC.append(cache, page, K, V, [2 * page + 5])
    rec = c[2, 1]
    assert rec[5 * 16:5 * 16 + 2].tolist() == [15 | (5 << 4), 9 | (8 << 4)]
    assert rec[page * 16 + 5 * 2:page * 16 + 5 * 2 + 2].view("<u2")[0] == 0x3F80
    half = page * 16 + page * 2
    assert rec[half + 5 * 16 + 15] == 8 | (15 << 4) and rec[half + page * 16 + 10:half + page * 16 + 12].view("<u2")[0] == 0x4000
    assert c[:2].sum() == 0
    k, v = KC.values(c, page, d)
    assert k[2, 1, 5, :4].tolist() == [7, -3, 1, 0] and v[2, 1, 5, 31] == 14


def test_non_finite_groups_are_stored_as_zeros():
    x = np.ones((1, 64))
    x[0, 3] = np.nan
    codes, s = KC.quantize(x)
    assert (codes[0, :32] == 8).all() and s[0, 0] == 2.0 ** -120 and (KC.dequantize(codes, s)[0, 32:] == 0.9375).all()


@pytest.mark.parametrize("interleaved", [0, 1])
def test_qk_norm_rope_against_torch_complex(interleaved):
    g = np.random.default_rng(2)
    x, gamma, cs = g.normal(size=(5, 3, 48)), g.uniform(0.5, 1.5, 48), KC.angles(50, 32)
    pos = np.array([0, 49, 7, -1, 3])
    y, _ = KC.qk_norm_rope(x, gamma, 1e-6, cs, pos, interleaved)
    t = torch.nn.functional.rms_norm(torch.from_numpy(x), (48,), torch.from_numpy(gamma), 1e-6)
    assert np.allclose(y[0], t[0].numpy()) and (y[3] == x[3]).all()       # position 0 turns nothing, -1 is padding
    a, b = (t[..., 0:32:2], t[..., 1:32:2]) if interleaved else (t[..., :16], t[..., 16:32])
    z = torch.complex(a, b) * torch.complex(*[torch.from_numpy(cs[np.maximum(pos, 0)].astype(np.float64))[:, None, i:i + 16] for i in (0, 16)])
    want = torch.stack([z.real, z.imag], -1).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)
    live = pos >= 0
    assert np.allclose(y[live][..., :32], want[live].numpy()) and np.allclose(y[live][..., 32:], t[live][..., 32:].numpy())


def _random_cache(g, pages, H, page, d):
    K, V = g.normal(size=(pages * page, H, d)), g.normal(size=(pages * page, H, d))
    b = lambda x: torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    cache = KC.append(np.zeros((pages, H, KC.record_bytes(page, d)), np.uint8), page, b(K), b(V), np.arange(pages * page))
    return cache


def test_attention_matches_the_dense_oracle_and_sdpa():
    g = np.random.default_rng(3)
    page, d, H = 16, 32, 2
    cache = _random_cache(g, 9, H, page, d)
    K, V = KC.values(cache, page, d)
    table, kv_len, offsets = np.array([[4, 0, 7], [8, 2, 1], [3, 5, 6]], np.int32), np.array([40, 0, 17]), np.array([0, 3, 5, 22])
    Q = g.normal(size=(22, 4, d))
    out, _ = KC.attention(Q, H, K, V, table, kv_len, offsets, page, 0.2, 0)
    assert (out[3:5] == 0).all()                      # no history: zeros
    for r in (0, 2):
        k = torch.from_numpy(K[table[r]]).permute(1, 0, 2, 3).reshape(H, -1, d)[:, :kv_len[r]]
        v = torch.from_numpy(V[table[r]]).permute(1, 0, 2, 3).reshape(H, -1, d)[:, :kv_len[r]]
        q = torch.from_numpy(Q[offsets[r]:offsets[r + 1]]).permute(1, 0, 2)
        for causal in (0, 1):
            n = q.shape[1]
            m = torch.arange(kv_len[r])[None] <= kv_len[r] - n + torch.arange(n)[:, None] if causal else None
            want = torch.nn.functional.scaled_dot_product_attention(q, k.repeat_interleave(2, 0), v.repeat_interleave(2, 0),
                                                                    attn_mask=m, scale=0.2)
            got, _ = KC.attention(Q, H, K, V, table, kv_len, offsets, page, 0.2, causal)
            assert np.allclose(got[offsets[r]:offsets[r + 1]], want.permute(1, 0, 2).numpy())


def test_attention_causal_rows_before_the_history_are_zero():
    g = np.random.default_rng(4)
    cache = _random_cache(g, 1, 1, 16, 32)
    K, V = KC.values(cache, 16, 32)
    out, _ = KC.attention(g.normal(size=(5, 1, 32)), 1, K, V, np.array([[0]]), [3], [0, 5], 16, 1.0, 1)
    assert (out[:2] == 0).all() and np.allclose(out[2, 0], V[0, 0, 0])


# ---- refusals -------------------------------------------------------------------------------------
@pytest.fixture(scope="module")
def rocs():
    from request_candidate_sharing_b200 import build
    build.build()
    from request_candidate_sharing_b200 import rocs as R
    return R


@pytest.fixture(scope="module")
def h(rocs):
    dummy = ctypes.create_string_buffer(256)      # refused before anything reads it as a handle
    yield ctypes.cast(dummy, ctypes.c_void_p)


def test_struct_layouts(rocs):
    assert ctypes.sizeof(rocs.Kv4Desc) == 16 and ctypes.sizeof(rocs.QkDesc) == 40
    assert rocs.QkDesc.eps.offset == 32 and rocs.QkDesc.io.offset == 36


@pytest.mark.parametrize("change", [dict(n_pages=0), dict(page_size=48), dict(page_size=256), dict(H_kv=0), dict(d_h=48), dict(d_h=256)])
def test_kv4_desc_refusals(rocs, h, change):
    d = rocs.Kv4Desc(**{**dict(n_pages=4, page_size=64, H_kv=8, d_h=32), **change})
    n = ctypes.c_size_t(0)
    assert rocs._lib_kv4_bytes(h, ctypes.byref(d), ctypes.byref(n)) == rocs.ROCS_ERR_INVALID_ARG
    assert rocs._lib_kv4_app(h, ctypes.byref(d), 16, 256, 16, 256, 16, 1, 16, None) == rocs.ROCS_ERR_INVALID_ARG
    assert rocs._lib_attn4_ws(h, ctypes.byref(d), 8, 1, 1, 1, ctypes.byref(n)) == rocs.ROCS_ERR_INVALID_ARG


def test_cache_bytes(rocs, h):
    n = ctypes.c_size_t(0)
    d = rocs.Kv4Desc(2000000, 128, 8, 128)
    assert rocs._lib_kv4_bytes(h, ctypes.byref(d), ctypes.byref(n)) == rocs.ROCS_OK
    assert n.value == 2000000 * 8 * KC.record_bytes(128, 128)       # past 32 bits


TAB = dict(past=1 << 20, new=2 << 20, B_R=4, page=16, free=3 << 20, n_free=8, n_pages=99, table=4 << 20, max_blocks=8, kv=5 << 20,
           off=6 << 20, slots=7 << 20, pos=8 << 20, rows=32, used=9 << 20, ws=None, ws_bytes=0)


@pytest.mark.parametrize("change,status", [
    (dict(new=None), 1), (dict(table=None), 1), (dict(kv=None), 1), (dict(off=None), 1), (dict(used=None), 1),
    (dict(slots=None), 1), (dict(pos=None), 1), (dict(B_R=0), 1), (dict(B_R=(1 << 24) + 1), 1), (dict(page=8), 1),
    (dict(page=65), 1), (dict(n_free=-1), 1), (dict(free=None), 1), (dict(n_pages=0), 1), (dict(max_blocks=0), 1),
    (dict(max_blocks=1 << 27), 1), (dict(rows=-1), 1), (dict(rows=(1 << 31) - 1), 1), (dict(slots=(7 << 20) + 8), 1),
    (dict(pos=(8 << 20) + 4), 1), (dict(kv=1 << 20), 1), (dict(kv=2 << 20), 1), (dict(off=(2 << 20) + 8), 1),
    (dict(kv=6 << 20), 1), (dict(used=(6 << 20) + 16), 1), (dict(table=3 << 20), 1), (dict(B_R=5000, table=64 << 20), 4),
])
def test_block_tables_refusals(rocs, h, change, status):
    a = {**TAB, **change}
    if a["B_R"] == 5000:
        a.update(past=1 << 24, new=2 << 24, kv=3 << 24, off=5 << 24)
    assert rocs._lib_tab(h, *a.values(), None) == status
    assert "rocs_kv_block_tables" in rocs.rocs_last_error()


def test_null_handles(rocs):
    assert rocs._lib_tab(None, *TAB.values(), None) == rocs.ROCS_ERR_INVALID_ARG
    d, q, n = rocs.Kv4Desc(4, 64, 8, 32), rocs.QkDesc(1, 1, 1, 32, 32, 0, 8, 1e-6, 1), ctypes.c_size_t(0)
    assert rocs._lib_qk(None, ctypes.byref(q), 16, 32, 16, 32, None, None, 16, 16, 16, 32, 16, 32, None) == 1
    assert rocs._lib_kv4_app(None, ctypes.byref(d), 16, 256, 16, 256, 16, 1, 16, None) == 1
    assert rocs._lib_kv4_get(None, ctypes.byref(d), 16, 16, 1, 16, 256, 16, 256, None) == 1
    assert rocs._lib_attn4(None, ctypes.byref(d), 16, 256, 8, 16, 16, 1, 16, 16, 1, 1, 1.0, 0, 16, 256, None, 0, None) == 1
    assert rocs._lib_attn4_ws(None, ctypes.byref(d), 8, 1, 1, 1, ctypes.byref(n)) == 1


QK = dict(rows=10, H_q=4, H_k=2, d_h=64, d_rot=64, interleaved=0, max_pos=100, eps=1e-6, io=1, Q=1 << 20, ld_Q=256, K=2 << 20, ld_K=128,
          gq=3 << 20, gk=4 << 20, cs=5 << 20, pos=6 << 20, Qo=7 << 20, ld_Qo=256, Ko=8 << 20, ld_Ko=128)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(rows=1 << 31), dict(H_q=-1), dict(H_q=0, H_k=0), dict(H_q=5000), dict(d_h=8), dict(d_h=264), dict(d_h=60),
    dict(d_rot=0), dict(d_rot=8), dict(d_rot=80), dict(d_rot=24), dict(interleaved=2), dict(max_pos=0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(io=2), dict(Q=None), dict(Ko=None), dict(cs=None), dict(pos=None),
    dict(ld_Q=255), dict(ld_Q=248), dict(ld_Ko=132), dict(Q=(1 << 20) + 2), dict(gq=(3 << 20) + 4), dict(cs=(5 << 20) + 8),
    dict(Qo=2 << 20), dict(Qo=(1 << 20) + 512), dict(Qo=1 << 20, ld_Qo=264), dict(Qo=8 << 20), dict(Ko=(1 << 20) + 1024, ld_Ko=256),
])
def test_qk_norm_rope_refusals(rocs, h, change):
    a = {**QK, **change}
    d = rocs.QkDesc(*[a[k] for k in ("rows", "H_q", "H_k", "d_h", "d_rot", "interleaved", "max_pos", "eps", "io")])
    st = rocs._lib_qk(h, ctypes.byref(d), *[a[k] for k in ("Q", "ld_Q", "K", "ld_K", "gq", "gk", "cs", "pos", "Qo", "ld_Qo", "Ko", "ld_Ko")], None)
    assert st == rocs.ROCS_ERR_INVALID_ARG and "rocs_qk_norm_rope" in rocs.rocs_last_error()


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(K=None), dict(V=None), dict(slots=None), dict(cache=None), dict(ld_K=248), dict(ld_V=260), dict(K=(1 << 20) + 8),
    dict(cache=(4 << 20) + 8), dict(slots=(3 << 20) + 4), dict(rows=(1 << 31) - 1),
])
def test_kv4_rows_refusals(rocs, h, change):
    a = {**dict(K=1 << 20, ld_K=256, V=2 << 20, ld_V=256, slots=3 << 20, rows=5, cache=4 << 20), **change}
    d = rocs.Kv4Desc(4, 64, 8, 32)
    assert rocs._lib_kv4_app(h, ctypes.byref(d), a["K"], a["ld_K"], a["V"], a["ld_V"], a["slots"], a["rows"], a["cache"], None) == 1
    assert rocs._lib_kv4_get(h, ctypes.byref(d), a["cache"], a["slots"], a["rows"], a["K"], a["ld_K"], a["V"], a["ld_V"], None) == 1


@pytest.mark.parametrize("change,append,gather", [
    (dict(K=4 << 20), 1, 1), (dict(V=(4 << 20) + 73712), 1, 1), (dict(cache=(1 << 20) + 2544), 1, 1), (dict(slots=(4 << 20) + 64), 1, 0),
    (dict(V=1 << 20), 0, 1), (dict(V=(1 << 20) + 512), 0, 1), (dict(ld_K=512, V=(1 << 20) + 512, ld_V=504), 0, 1), (dict(slots=(1 << 20) + 80), 0, 1),
])
def test_kv4_rows_overlaps_are_refused(rocs, h, change, append, gather):
    a = {**dict(K=1 << 20, ld_K=256, V=2 << 20, ld_V=256, slots=3 << 20, rows=5, cache=4 << 20), **change}
    d = rocs.Kv4Desc(4, 64, 8, 32)             # 73728 bytes
    if append:
        assert rocs._lib_kv4_app(h, ctypes.byref(d), a["K"], a["ld_K"], a["V"], a["ld_V"], a["slots"], a["rows"], a["cache"], None) == 1
        assert "overlaps" in rocs.rocs_last_error()
    if gather:
        assert rocs._lib_kv4_get(h, ctypes.byref(d), a["cache"], a["slots"], a["rows"], a["K"], a["ld_K"], a["V"], a["ld_V"], None) == 1
        assert "overlap" in rocs.rocs_last_error()


AT = dict(Q=1 << 20, ld_Q=512, H_q=16, cache=2 << 20, table=3 << 20, max_blocks=4, kv=4 << 20, off=5 << 20, B_R=2, rows=7, scale=0.125,
          causal=0, O=6 << 20, ld_O=512, ws=None, ws_bytes=0)


@pytest.mark.parametrize("change", [
    dict(Q=None), dict(cache=None), dict(table=None), dict(kv=None), dict(off=None), dict(O=None), dict(H_q=12), dict(H_q=0), dict(ld_Q=504),
    dict(ld_O=516), dict(Q=(1 << 20) + 8), dict(O=(6 << 20) + 8), dict(cache=(2 << 20) + 8), dict(B_R=0), dict(B_R=1 << 25), dict(rows=-1),
    dict(rows=1 << 28), dict(rows=(2 ** 31 - 255) // 16 + 1), dict(B_R=1 << 24, rows=1, H_q=64, ld_Q=2048, ld_O=2048, H_kv=64), dict(max_blocks=0),
    dict(kv=(4 << 20) + 2), dict(off=(5 << 20) + 1), dict(table=(3 << 20) + 2),
    dict(max_blocks=1 << 25), dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=2),
])
def test_attention_refusals(rocs, h, change):
    d = rocs.Kv4Desc(40, 64, change.get("H_kv", 8), 32)
    assert rocs._lib_attn4(h, ctypes.byref(d), *{**AT, **{k: v for k, v in change.items() if k != "H_kv"}}.values(), None) == rocs.ROCS_ERR_INVALID_ARG
    assert "rocs_dca_cross_attn_kv4" in rocs.rocs_last_error()


# ---- pages that run out -----------------------------------------------------------------------------
def test_block_tables_requests_behind_one_that_does_not_fit():
    # pages of 16, three free: 20 tokens take two, 70 would take five and get none, 1 takes the third, 5 find nothing
    table = np.full((4, 5), -1, np.int32)
    t, kv, off, slots, pos, used, st = KC.block_tables(None, [20, 70, 1, 5], 16, [8, 3, 6], 10, table, 96)
    assert kv.tolist() == [20, 0, 1, 0] and off.tolist() == [0, 20, 90, 91, 96] and used == 3 and st == {"counts"}
    assert t[:, :2].tolist() == [[8, 3], [-1, -1], [6, -1], [-1, -1]] and (t[:, 2:] == -1).all()
    assert slots[:20].tolist() == [*range(128, 144), *range(48, 52)] and slots[90] == 96 and pos[90] == 0
    assert (slots[20:90] == -1).all() and (slots[91:] == -1).all() and (pos[20:90] == -1).all() and (pos[91:] == -1).all()


@pytest.mark.parametrize("scale", [1.01 * 2.0 ** 126, -1.01 * 2.0 ** 126])
def test_attention_refuses_scales_whose_products_overflow(rocs, h, scale):
    d = rocs.Kv4Desc(40, 64, 8, 32)
    assert rocs._lib_attn4(h, ctypes.byref(d), *{**AT, "scale": scale}.values(), None) == rocs.ROCS_ERR_INVALID_ARG
    assert "2^126" in rocs.rocs_last_error()


@pytest.mark.parametrize("change", [      # Qo is 10 rows of 512 bytes, Ko of 256
    dict(Qo=(3 << 20) + 240), dict(Qo=(4 << 20) - 5104), dict(Ko=(3 << 20) + 240), dict(Ko=(4 << 20) - 2544), dict(Qo=(5 << 20) + 25584),
    dict(Ko=(5 << 20) - 2544), dict(Qo=(6 << 20) + 32), dict(Ko=6 << 20), dict(Ko=(6 << 20) - 4592, ld_Ko=256), dict(H_q=0, Ko=4 << 20),
])
def test_qk_norm_rope_refuses_outputs_over_its_tables(rocs, h, change):
    a = {**QK, **change}
    d = rocs.QkDesc(*[a[k] for k in ("rows", "H_q", "H_k", "d_h", "d_rot", "interleaved", "max_pos", "eps", "io")])
    st = rocs._lib_qk(h, ctypes.byref(d), *[a[k] for k in ("Q", "ld_Q", "K", "ld_K", "gq", "gk", "cs", "pos", "Qo", "ld_Qo", "Ko", "ld_Ko")], None)
    assert st == rocs.ROCS_ERR_INVALID_ARG and "overlaps the gammas, the angles or the positions" in rocs.rocs_last_error()


@pytest.mark.parametrize("at,what", [("past", "input"), ("new", "input"), ("free", "input"), ("table", "output"), ("kv", "output"), ("off", "output"),
                                     ("slots", "output"), ("pos", "output"), ("used", "output")])
def test_block_tables_refuses_a_workspace_over_its_tensors(rocs, h, at, what):
    a = {**TAB, "B_R": 5000, **{k: (i + 1) << 24 for i, k in enumerate(("past", "new", "free", "table", "kv", "off", "slots", "pos", "used"))}}
    n = ctypes.c_size_t(0)
    assert rocs._lib_tab_ws(h, 5000, ctypes.byref(n)) == rocs.ROCS_OK and n.value > 16
    a.update(ws=a[at] - n.value + 16, ws_bytes=n.value)
    a["ws"] -= a["ws"] % 16
    assert rocs._lib_tab(h, *a.values(), None) == rocs.ROCS_ERR_INVALID_ARG
    assert f"the workspace overlaps an {what}" in rocs.rocs_last_error()


@pytest.mark.parametrize("at", ["past", "new", "free", "table", "kv", "off", "used"])
def test_block_tables_refuses_misaligned_tensors(rocs, h, at):
    assert rocs._lib_tab(h, *{**TAB, at: TAB[at] + 2}.values(), None) == rocs.ROCS_ERR_INVALID_ARG
    assert "misaligned" in rocs.rocs_last_error()
