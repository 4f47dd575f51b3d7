"""Appends with the rotary embedding into paged caches, in the cache's type and
in 8 bits, against the fp64 restatement in tests/q8_ref.py (GPU only)."""
from __future__ import annotations

import numpy as np
import pytest

from tests import q8_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def loki(cuda):
    import sparse_attention_decode_loki_b200 as m
    return m


def make(torch, dev, B, H_kv, G, T, D, page, pos, new, dt, basis, rot, d_lo, block, seed, n_pos=None,
         spare=2):
    """Inputs on the device: random rows and pool, shuffled pages for every touched place."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    need = [range(p // page, -(-(p + n) // page) if n else p // page) for p, n in zip(pos, new)]
    n_pages = max(1, sum(len(r) for r in need) + spare)
    order = torch.randperm(n_pages, generator=g).tolist()
    width = max(1, max((r.stop for r in need)))
    bt = torch.full((B, width), -1, dtype=torch.int32)
    for b, r in enumerate(need):
        for lp in r:
            bt[b, lp] = order.pop()
    s = dict(
        K=rnd(B, H_kv, T, D).to(dt), V=(rnd(B, H_kv, T, D) * 0.7).to(dt),
        q=rnd(B, H_kv * G, T, D).to(dt),
        P=torch.linalg.qr(rnd(H_kv, D, D))[0].contiguous() if basis else None,
        bt=bt, pos=torch.tensor(pos, dtype=torch.int32), new=torch.tensor(new, dtype=torch.int32),
        lo=rnd(n_pages, H_kv, page, d_lo).to(dt) if d_lo else None)
    if block:
        s["Kp"] = (rnd(n_pages, H_kv, page, D) * 60).to(torch.float8_e4m3fn)
        s["Vp"] = (rnd(n_pages, H_kv, page, D) * 60).to(torch.float8_e4m3fn)
        # scales well below, around and above what the new rows need
        e = torch.randint(-12, -4, (2, n_pages, H_kv, page // block), generator=g)
        s["ks"], s["vs"] = torch.exp2(e[0].float()), torch.exp2(e[1].float())
    else:
        s["Kp"], s["Vp"] = rnd(n_pages, H_kv, page, D).to(dt), rnd(n_pages, H_kv, page, D).to(dt)
    return {k: v.to(dev).contiguous() if hasattr(v, "to") else v for k, v in s.items()}


def table_for(loki, dev, n_pos, rot):
    return loki.loki_rope_table(n_pos, rot, device=dev) if rot else None


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def half_step(torch, dt):
    return torch.finfo(dt).eps / 2


def check_rows(torch, got, want, dt, bound):
    """fp32 arithmetic off by at most `bound`, then one rounding to dt."""
    tol = half_step(torch, dt) * (np.abs(want) + bound) + bound
    assert np.all(np.abs(got - want) <= tol), np.abs(got - want).max()


def row_bound(x, rows, P):
    """fp32 error of a key row: the rotary embedding's products and sum (3 roundings of at most
    |a| + |b|, cos and sin given), then D products summed with the basis."""
    r = 4 * 2.0 ** -24 * 2 * np.abs(x).max(-1, keepdims=True)
    if P is None:
        return np.broadcast_to(r, rows.shape)
    n = x.shape[-1]
    return (np.abs(rows) * 0 + r * np.abs(P).sum(-2)
            + (n + 2) * 2.0 ** -24 * (2 * np.abs(x).max(-1, keepdims=True) * np.abs(P).sum(-2)))


def expect(s, table, inter):
    """Exact rotated queries and keys (fp64) and the keys' fp32 error bounds."""
    K, q, P = f64(s["K"]), f64(s["q"]), f64(s["P"])
    pos = s["pos"].cpu().numpy()
    T = K.shape[2]
    Kr, qr, bound = np.empty_like(K), np.empty_like(q), np.empty_like(K)
    for b in range(K.shape[0]):
        j = np.minimum(pos[b] + np.arange(T), (len(table) if table is not None else 1 << 30) - 1)
        qr[b] = q8_ref.rope(q[b], j, table, inter)
        for h in range(K.shape[1]):
            x = q8_ref.rope(K[b, h], j, table, inter)
            Kr[b, h] = x @ P[h] if P is not None else x
            bound[b, h] = row_bound(K[b, h], Kr[b, h], P[h] if P is not None else None)
    return Kr, qr, bound


def places(s, page):
    """(b, t, page, slot) of every appended token."""
    bt, pos, new = (s[k].cpu().numpy() for k in ("bt", "pos", "new"))
    return [(b, t, int(bt[b, (pos[b] + t) // page]), int((pos[b] + t) % page))
            for b in range(len(pos)) for t in range(new[b])]


CASES = [
    # B, H_kv, G, T, D, page, pos, new, dtype, basis, rot, interleaved, d_lo, block
    (2, 3, 1, 1, 128, 16, [0, 77], [1, 1], "bf16", True, 128, False, 32, 16),
    (3, 2, 4, 5, 128, 32, [30, 0, 63], [5, 0, 3], "bf16", True, 64, True, 16, 32),
    (1, 1, 1, 1, 128, 128, [511], [1], "f32", True, 128, False, 0, 128),
    (2, 2, 2, 70, 96, 64, [15, 200], [70, 41], "bf16", True, 96, False, 32, 64),
    (2, 5, 1, 33, 96, 48, [1, 47], [33, 1], "f32", True, 48, True, 20, 16),
    (1, 2, 3, 300, 128, 64, [129], [300], "bf16", True, 128, False, 32, 16),
    (1, 2, 1, 300, 128, 256, [5], [300], "bf16", False, 128, True, 0, 128),
    (4, 2, 8, 17, 128, 16, [3, 16, 31, 100], [17, 1, 16, 9], "bf16", False, 0, False, 64, 16),
    (2, 1, 5, 130, 128, 128, [0, 127], [130, 129], "f32", False, 32, False, 16, 64),
    (9, 2, 1, 1, 128, 64, [0, 1, 15, 16, 63, 64, 100, 5, 6], [1, 1, 1, 0, 1, 1, 1, 1, 1], "bf16", True,
     128, False, 64, 32),
    (40, 4, 2, 2, 128, 32, list(range(40)), [2] * 40, "bf16", True, 128, False, 32, 32),
    (1, 8, 4, 1000, 128, 64, [64], [1000], "bf16", True, 128, False, 16, 64),
]


def ids(c):
    return "B%d-H%d-T%d-D%d-p%d-%s-%s-r%d%s-blk%d" % (c[0], c[1], c[3], c[4], c[5], c[8],
                                                    "P" if c[9] else "noP", c[10], "i" if c[11] else "", c[13])


def dtype(torch, name):
    return torch.bfloat16 if name == "bf16" else torch.float32


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_append_rope_matches_formula(loki, cuda, case):
    import torch
    B, H, G, T, D, page, pos, new, dtn, basis, rot, inter, d_lo, _ = case
    dt = dtype(torch, dtn)
    s = make(torch, cuda, B, H, G, T, D, page, pos, new, dt, basis, rot, d_lo, 0, 11)
    tab = table_for(loki, cuda, max(pos) + T, rot)
    before = {k: s[k].clone() for k in ("Kp", "Vp", "lo") if s[k] is not None}
    q_out = torch.full_like(s["q"], 7.0)
    got = loki.loki_append_keys_paged_rope(s["K"], s["V"], s["P"], s["Kp"], s["Vp"], s["bt"], s["pos"],
                                           rope_table=tab, interleaved=inter, Kt_lo_pages=s["lo"],
                                           new_lens=s["new"], q=s["q"], q_out=q_out)
    assert got is q_out
    torch.cuda.synchronize()
    assert loki.loki_device_error(reset=True) == 0
    Kr, qr, bound = expect(s, f64(tab), inter)
    Kg, Vg, lo, qg = f64(s["Kp"]), f64(s["Vp"]), f64(s["lo"]), f64(q_out)
    want_K, want_V = f64(before["Kp"]), f64(before["Vp"])
    touched = np.zeros(want_K.shape[:3], bool)
    for b, t, p, slot in places(s, page):
        check_rows(torch, Kg[p, :, slot], Kr[b, :, t], dt, bound[b, :, t])
        assert np.array_equal(Vg[p, :, slot], f64(s["V"])[b, :, t])
        if lo is not None:
            assert np.array_equal(lo[p, :, slot], Kg[p, :, slot, :d_lo])
        touched[p, :, slot] = True
    assert np.array_equal(Kg[~touched], want_K[~touched]) and np.array_equal(Vg[~touched], want_V[~touched])
    if lo is not None:
        assert np.array_equal(lo[~touched], f64(before["lo"])[~touched])
    for b in range(B):
        check_rows(torch, qg[b, :, : new[b]], qr[b, :, : new[b]], dt,
                   8 * 2.0 ** -24 * np.abs(f64(s["q"])[b, :, : new[b]]).max(-1, keepdims=True, initial=0))
        assert np.all(qg[b, :, new[b]:] == 7.0)


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_append_q8_matches_formula(loki, cuda, case):
    import torch
    B, H, G, T, D, page, pos, new, dtn, basis, rot, inter, d_lo, block = case
    dt = dtype(torch, dtn)
    s = make(torch, cuda, B, H, G, T, D, page, pos, new, dt, basis, rot, d_lo, block, 12)
    tab = table_for(loki, cuda, max(pos) + T, rot)
    names = ("Kp", "Vp", "ks", "vs")
    before = {k: f64(s[k]) for k in names}
    lo_before = f64(s["lo"])
    q_out = loki.loki_append_keys_paged_q8(s["K"], s["V"], s["P"], s["Kp"], s["Vp"], s["ks"], s["vs"],
                                           s["bt"], s["pos"], rope_table=tab, interleaved=inter,
                                           Kt_lo_pages=s["lo"], new_lens=s["new"], q=s["q"])
    torch.cuda.synchronize()
    assert loki.loki_device_error(reset=True) == 0
    Kr, qr, bound = expect(s, f64(tab), inter)
    got = {k: f64(s[k]) for k in names}
    want = {k: v.copy() for k, v in before.items()}
    tol = {k: np.zeros_like(want[k]) for k in ("Kp", "Vp")}
    bt = s["bt"].cpu().numpy()
    for b in range(B):
        for h in range(H):
            for lo, hi in spans(pos[b], new[b], block):
                p, at = bt[b, lo // page], lo % page // block
                sl = slice(at * block, (at + 1) * block)
                for nm, sc, rows, bd in (("Kp", "ks", Kr, bound), ("Vp", "vs", f64(s["V"]), None)):
                    x = rows[b, h, lo - pos[b]:hi - pos[b]]
                    first = lo % block
                    codes, scale = q8_ref.append_block(want[nm][p, h, sl], want[sc][p, h, at], x, first)
                    if bd is not None:  # values are exact; a key's amax must not hang on its last bits
                        top = np.abs(x).max()
                        assert abs(top / (448 * q8_ref.pow2_scale(top)) - 1) > 1e-5
                        assert abs(top / (224 * q8_ref.pow2_scale(top)) - 1) > 1e-5
                    want[nm][p, h, sl], want[sc][p, h, at] = codes, scale
                    if bd is not None:  # fp32 arithmetic may land on the code next to the exact value's
                        y = x / scale
                        bb = bd[b, h, lo - pos[b]:hi - pos[b]] / scale
                        lo_c, hi_c = q8_ref.e4m3_round(y - bb), q8_ref.e4m3_round(y + bb)
                        w = want[nm][p, h, sl][first:first + len(x)]
                        tol[nm][p, h, sl][first:first + len(x)] = np.maximum(np.abs(lo_c - w), np.abs(hi_c - w))
    for k in ("ks", "vs"):
        assert np.array_equal(got[k], want[k]), k
    for k in ("Kp", "Vp"):
        assert np.all(np.abs(got[k] - want[k]) <= tol[k]), k
    if s["lo"] is not None:
        lo = f64(s["lo"])
        touched = np.zeros(lo.shape[:3], bool)
        for b, t, p, slot in places(s, page):
            check_rows(torch, lo[p, :, slot], Kr[b, :, t, :d_lo], dt, bound[b, :, t, :d_lo])
            touched[p, :, slot] = True
        assert np.array_equal(lo[~touched], lo_before[~touched])
    qg = f64(q_out)
    for b in range(B):
        check_rows(torch, qg[b, :, : new[b]], qr[b, :, : new[b]], dt,
                   8 * 2.0 ** -24 * np.abs(f64(s["q"])[b, :, : new[b]]).max(-1, keepdims=True, initial=0))


def spans(p0, n, block):
    """The appended tokens [p0, p0 + n) cut at block borders."""
    out, lo = [], p0
    while lo < p0 + n:
        hi = min(p0 + n, (lo // block + 1) * block)
        out.append((lo, hi))
        lo = hi
    return out


@pytest.mark.parametrize("q8", [False, True], ids=["dt", "q8"])
def test_defaults_append_all_tokens_without_tables(loki, cuda, q8):
    """No rope table, basis, plane, queries or new_lens: rows go in as they are."""
    import torch
    s = make(torch, cuda, 2, 2, 1, 20, 128, 32, [0, 32], [20, 20], torch.bfloat16, False, 0, 0,
             16 if q8 else 0, 13)
    if q8:
        r = loki.loki_append_keys_paged_q8(s["K"], s["V"], None, s["Kp"], s["Vp"], s["ks"], s["vs"], s["bt"], s["pos"])
    else:
        r = loki.loki_append_keys_paged_rope(s["K"], s["V"], None, s["Kp"], s["Vp"], s["bt"], s["pos"])
    assert r is None
    sc = s["ks"].repeat_interleave(16, dim=2)[..., None] if q8 else 1.0
    for b, t, p, slot in places(s, 32):
        have = (s["Kp"].float() * sc)[p, :, slot].double().cpu().numpy()
        want = s["K"][b, :, t].double().cpu().numpy()
        top = np.abs(want).max()
        assert np.all(np.abs(have - want) <= (np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -17 * top * 64) if q8 else 0))
        if not q8:
            assert torch.equal(s["Vp"][p, :, slot], s["V"][b, :, t])
    assert loki.loki_device_error(reset=True) == 0


def test_rope_table_matches_fp64(loki, cuda):
    for n, r, base, ps in ((1, 16, 10000.0, 1.0), (5000, 128, 10000.0, 1.0), (70001, 64, 500000.0, 0.25)):
        t = f64(loki.loki_rope_table(n, r, base, ps, device=cuda))
        ang = np.arange(n)[:, None] * ps * base ** (-2.0 * np.arange(r // 2) / r)
        want = np.concatenate([np.cos(ang), np.sin(ang)], axis=1)
        # one rounding to fp32, and the angle's own 64-bit rounding
        assert np.all(np.abs(t - want) <= 2.0 ** -24 * np.abs(want) + 1e-10)


def test_append_queries_in_place(loki, cuda):
    import torch
    for inter in (False, True):
        s = make(torch, cuda, 3, 2, 4, 9, 128, 16, [0, 5, 40], [9, 9, 9], torch.bfloat16, False, 128, 0, 0, 14)
        tab = table_for(loki, cuda, 64, 128)
        args = (s["K"], s["V"], None, s["Kp"], s["Vp"], s["bt"], s["pos"])
        apart = loki.loki_append_keys_paged_rope(*args, rope_table=tab, interleaved=inter, q=s["q"])
        loki.loki_append_keys_paged_rope(*args, rope_table=tab, interleaved=inter, q=s["q"], q_out=s["q"])
        assert torch.equal(apart, s["q"])


def test_q8_step_by_step_gives_the_prompts_scales(loki, cuda):
    """Tokens appended one at a time end with the block scales of one append, and codes at most one
    requantisation step apart (two roundings instead of one where a code fell among the subnormals)."""
    import torch
    T, page, block = 50, 32, 16
    s = make(torch, cuda, 1, 2, 1, T, 128, page, [0], [T], torch.bfloat16, True, 128, 0, block, 15)
    s["K"] *= torch.linspace(0.1, 8, T, device=cuda).to(torch.bfloat16)[:, None]
    tab = table_for(loki, cuda, T, 128)
    keep = {k: s[k].clone() for k in ("Kp", "Vp", "ks", "vs")}
    loki.loki_append_keys_paged_q8(s["K"], s["V"], s["P"], s["Kp"], s["Vp"], s["ks"], s["vs"], s["bt"],
                                   s["pos"], rope_table=tab)
    for t in range(T):
        loki.loki_append_keys_paged_q8(s["K"][:, :, t:t + 1].contiguous(), s["V"][:, :, t:t + 1].contiguous(),
                                       s["P"], keep["Kp"], keep["Vp"], keep["ks"], keep["vs"], s["bt"],
                                       torch.tensor([t], dtype=torch.int32, device=cuda), rope_table=tab)
    used = [int(p) for p in s["bt"][0].cpu()]
    for c, sc in (("Kp", "ks"), ("Vp", "vs")):
        nb = page // block
        for i in range(-(-T // block)):
            p, at = used[i * block // page], i % nb
            assert torch.equal(s[sc][p, :, at], keep[sc][p, :, at])
            n = min(block, T - i * block)
            a, b = (x[c][p, :, at * block:at * block + n].float() for x in (s, keep))
            # equal outside the subnormals (|code| < 2^-6); there two roundings, each at most half of 2^-9
            assert torch.all(((a - b).abs() <= 2.0 ** -9) | (a == b))
            # kernels of few and of many rows may round fp32 sums differently: one code step at most
            big = a.abs() >= 2.0 ** -6
            assert torch.all((a - b)[big].abs() <= 2.0 ** -3 * a[big].abs())


def test_q8_reused_page_starts_afresh_and_zero_rows(loki, cuda):
    """A block whose first row is appended ignores its page's old scale; all-zero blocks are zeros."""
    import torch
    s = make(torch, cuda, 1, 1, 1, 16, 128, 16, [0], [16], torch.bfloat16, False, 0, 0, 16, 16)
    s["ks"].fill_(float("nan"))
    s["vs"].fill_(2.0 ** 100)
    s["K"].zero_()
    loki.loki_append_keys_paged_q8(s["K"], s["V"], None, s["Kp"], s["Vp"], s["ks"], s["vs"], s["bt"], s["pos"])
    p = int(s["bt"][0, 0])
    assert float(s["ks"][p, 0, 0]) == 2.0 ** -126 and torch.all(s["Kp"][p].float() == 0)
    assert float(s["vs"][p, 0, 0]) == q8_ref.pow2_scale(float(s["V"].abs().max()))


def test_q8_infinities_saturate_and_nan_stays(loki, cuda):
    import torch
    s = make(torch, cuda, 1, 1, 1, 4, 128, 16, [0], [4], torch.float32, False, 0, 0, 16, 17)
    s["K"][0, 0, 0, 3], s["K"][0, 0, 1, 5], s["K"][0, 0, 2, 7] = float("inf"), float("-inf"), float("nan")
    loki.loki_append_keys_paged_q8(s["K"], s["V"], None, s["Kp"], s["Vp"], s["ks"], s["vs"], s["bt"], s["pos"])
    p = int(s["bt"][0, 0])
    K = s["Kp"][p, 0].float().cpu()
    fin = s["K"][torch.isfinite(s["K"])].abs().max()
    assert float(s["ks"][p, 0, 0]) == q8_ref.pow2_scale(float(fin))
    assert K[0, 3] == 448 and K[1, 5] == -448 and torch.isnan(K[2, 7])
    assert int(torch.isnan(K[:4]).sum()) == 1


@pytest.mark.parametrize("q8", [False, True], ids=["dt", "q8"])
def test_tokens_without_a_place_are_left_out_and_flagged(loki, cuda, q8):
    """Bad pages, positions behind the block table and behind the rope table: the other tokens go in."""
    import torch
    block = 16 if q8 else 0

    def fresh(pos, seed=18):
        s = make(torch, cuda, 2, 1, 1, 20, 128, 16, pos, [20, 20], torch.bfloat16, False, 128, 0, block, seed)
        return s, s["Kp"].clone()

    def run(s, tab):
        a = (s["K"], s["V"], None, s["Kp"], s["Vp"])
        f = loki.loki_append_keys_paged_q8 if q8 else loki.loki_append_keys_paged_rope
        f(*a, *((s["ks"], s["vs"]) if q8 else ()), s["bt"], s["pos"], rope_table=tab)
        torch.cuda.synchronize()
        return loki.loki_device_error(reset=True)

    def same(s, old, p):
        return torch.equal(s["Kp"].view(torch.uint8)[p], old.view(torch.uint8)[p])

    tab = table_for(loki, cuda, 64, 128)
    for bad in (-1, 1 << 20):
        s, old = fresh([0, 16])
        gone = int(s["bt"][0, 1])
        s["bt"][0, 1] = bad
        assert run(s, tab) == 2
        assert same(s, old, gone) and not same(s, old, int(s["bt"][0, 0])) and not same(s, old, int(s["bt"][1, 1]))
    s, old = fresh([0, 16])
    assert run(s, tab[:30].contiguous()) == 3
    last = int(s["bt"][1, 2])  # tokens 32.. of sequence 1: behind the table
    assert same(s, old, last) and not same(s, old, int(s["bt"][1, 1]))
    s, old = fresh([0, 16])
    s["pos"][1] = 40  # tokens 48.. lie behind the block table
    s["bt"][1, 2] = int(s["bt"][1, 1])
    assert run(s, tab) == 2
    s, old = fresh([0, 16])
    s["pos"][0] = -30  # tokens before the sequence's start
    assert run(s, tab) == 2


def test_append_on_another_stream_and_in_a_graph(loki, cuda):
    import torch
    s = make(torch, cuda, 2, 2, 2, 3, 128, 16, [14, 3], [3, 3], torch.bfloat16, True, 128, 32, 16, 19)
    tab = table_for(loki, cuda, 32, 128)
    q_out = torch.empty_like(s["q"])
    names = ("Kp", "Vp", "ks", "vs", "lo")
    start = {k: s[k].clone() for k in names}

    def call():
        loki.loki_append_keys_paged_q8(s["K"], s["V"], s["P"], s["Kp"], s["Vp"], s["ks"], s["vs"], s["bt"],
                                       s["pos"], rope_table=tab, Kt_lo_pages=s["lo"], q=s["q"], q_out=q_out)

    call()
    want = {k: s[k].clone() for k in names}
    wq = q_out.clone()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        call()
    for _ in range(2):
        for k in names:
            s[k].copy_(start[k])
        q_out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s[k].view(torch.uint8), want[k].view(torch.uint8)) for k in names)
        assert torch.equal(q_out, wq)
