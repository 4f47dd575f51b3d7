"""Measured cases of the paged cache with rotary appends and 8-bit storage.

Four operators: the append with the rotary embedding into pages of the input
type ("append"), the same append into pages held in 8 bits with one power-of-two
scale for each block of tokens and KV head ("append8"), attention of one query
token per sequence over the whole 8-bit cache ("dense8"), and attention over
each query head's selected tokens of that cache ("sparse8").

`run` computes them with elementary torch operations where `own` is false and
with this repository's entry points where it is true.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_F8 = torch.float8_e4m3fn
_SIZE = {"bf16": 2, "f32": 4}


def _lib():
    import sparse_attention_decode_loki_b200 as loki
    return loki


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    mha13 = dict(H_q=40, H_kv=40, D=128, dt="bf16")
    mha7 = dict(H_q=32, H_kv=32, D=128, dt="bf16")
    gqa = dict(H_q=32, H_kv=8, D=128, dt="bf16")
    rot = dict(rot_dim=128, interleaved=False)
    return [
        # one token for each of 16 sequences, Llama2-13B heads: the append of every decode step
        dict(name="append-step-13b", op="append", B=16, T=1, at=4095, basis=True, d_lo=32, page=64, **mha13, **rot),
        # a ragged batch of prompts behind cached prefixes, Llama-3-8B heads
        dict(name="append-prompts-gqa", op="append", B=4, T=2048, at=500, basis=True, d_lo=16, page=64, **gqa, **rot),
        # the same decode step's append into the 8-bit cache
        dict(name="append8-step-13b", op="append8", B=16, T=1, at=4095, basis=True, d_lo=32, page=64, block=16, **mha13, **rot),
        # one prompt of 4096 tokens, Llama2-7B heads, into the 8-bit Loki cache
        dict(name="append8-prompt-7b", op="append8", B=1, T=4096, at=0, basis=True, d_lo=32, page=64, block=32, **mha7, **rot),
        # prompts into an 8-bit cache for dense attention alone (no basis, no plane)
        dict(name="append8-prompts-gqa-plain", op="append8", B=2, T=8192, at=77, basis=False, d_lo=0, page=128, block=64, **gqa, **rot),
        # a short chat, one sequence: latency
        dict(name="dense8-short-7b", op="dense8", B=1, S=513, page=16, block=16, **mha7),
        # ragged batch at the Llama2-13B decode shape
        dict(name="dense8-ragged-13b", op="dense8", B=16, S=4096, page=64, block=16, **mha13),
        # long contexts with grouped heads, Llama-3-8B
        dict(name="dense8-long-gqa", op="dense8", B=4, S=32768, page=64, block=32, **gqa),
        # Loki's last step for one sequence, a quarter of 4096 tokens selected
        dict(name="sparse8-7b", op="sparse8", B=1, S=4096, k=1024, page=64, block=16, **mha7),
        # the batched decode, an eighth selected
        dict(name="sparse8-ragged-13b", op="sparse8", B=16, S=4096, k=512, page=64, block=16, **mha13),
        # long contexts, a sixteenth selected
        dict(name="sparse8-long-gqa", op="sparse8", B=4, S=32768, k=2048, page=64, block=32, **gqa),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    """Head counts, lengths, pages and types over the whole ranges, at most the largest listed work."""
    op = rng.choice(["append", "append8", "dense8", "sparse8"])
    G = rng.choice([1, 1, 2, 3, 4, 5, 8])
    H_kv = rng.choice([1, 2, 4, 5, 8, 8]) if G > 1 else rng.choice([1, 3, 8, 12, 32, 40])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    block = rng.choice([b for b in (16, 32, 64, 128) if page % b == 0])
    D = rng.choice([128, 128, 128, 96])
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    c = dict(op=op, H_q=G * H_kv, H_kv=H_kv, D=D, dt=dt, page=page)
    if op in ("append", "append8"):
        # at most 2^17 (token, KV head) rows and as many query rows: as the listed prompts
        c["T"] = 1 if rng.random() < 0.4 else _log(rng, 2, 8192)
        c["B"] = _log(rng, 1, max(1, min(64, (1 << 17) // (c["T"] * G * H_kv))))
        c["T"] = max(1, min(c["T"], (1 << 17) // (c["B"] * G * H_kv)))
        c["at"] = _log(rng, 1, 30000) - 1
        c["basis"] = rng.random() < 0.7
        c["d_lo"] = rng.choice([0, 16, 32, 64])
        c["rot_dim"] = rng.choice([D, D, D // 2])
        c["interleaved"] = rng.random() < 0.3
        if op == "append8":
            c["block"] = block
        return c
    # at most 2^20 (token, KV head) rows: as the listed long contexts
    c["S"] = _log(rng, 1, 32768)
    c["B"] = _log(rng, 1, max(1, min(64, (1 << 20) // (c["S"] * H_kv))))
    c["block"] = block
    if op == "sparse8":
        # at most 2^18 selected (token, query head) rows
        c["k"] = max(1, min(c["S"], int(c["S"] * rng.choice([0.05, 0.125, 0.25, 1.0])), (1 << 18) // (c["B"] * G * H_kv)))
    return c


def _lens(case):
    """The sequences' lengths of an attention case (or their new tokens', of an append): from full down to a
    few tokens, one empty sequence where there are at least six. Part of the case, so not of the seed."""
    B, n = case["B"], case.get("S", case.get("T"))
    if B == 1 or n == 1:
        return [n] * B
    lens = [max(1, n - (n * b) // (2 * B)) for b in range(B)]
    if B >= 6:
        lens[1], lens[2] = 0, max(1, n // 37)
    return lens


def _positions(case):
    """The first appended token's index of each sequence: no two at the same place of a page."""
    return [max(0, case["at"] - 37 * b) for b in range(case["B"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _basis(g, H, D):
    return torch.linalg.qr(_rand(g, H, D, D).double())[0].float().contiguous()


def _keys(g, n, H, D, basis):
    """Keys of decaying spectrum in a basis per head, as PCA finds them: [n, H, D]."""
    sig = torch.exp(-torch.arange(D, device="cuda", dtype=torch.float32) / 20.0)
    return torch.matmul((_rand(g, n, H, 1, D) * sig), basis.transpose(-1, -2)).squeeze(2) + 0.01 * _rand(g, n, H, D)


def _rope_angles(n_pos, rot_dim):
    inv = 10000.0 ** (-2.0 * torch.arange(rot_dim // 2, dtype=torch.float64, device="cuda") / rot_dim)
    ang = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()


def _pow2_scale(amax):
    """The least power of two s (at least 2^-126) with amax <= 448 s."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(min=-126)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, -126)))


def _tables(case, pages, g):
    """A block table whose sequence b has pages[b] (first, last) pages of its own in a shuffled pool, three spare
    pages, and -1 where a sequence has none."""
    B = case["B"]
    total = sum(max(0, b - a) for a, b in pages)
    n_pages = total + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(b for _, b in pages))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, (first, last) in enumerate(pages):
        table[b, first:last] = order[at:at + max(0, last - first)]
        at += max(0, last - first)
    return table, n_pages


def _prepare_append(case, g):
    B, T, H_q, H_kv, D, page = (case[k] for k in ("B", "T", "H_q", "H_kv", "D", "page"))
    dt = _DT[case["dt"]]
    new, pos = _lens(case), _positions(case)
    # the pool holds the pages that the append touches (older ones are never read), each with tokens in it already
    pages = [(p // page, -(-(p + n) // page) if n else p // page) for p, n in zip(pos, new)]
    table, n_pages = _tables(case, pages, g)
    R = _basis(g, H_kv, D)
    rows = _keys(g, B * T, H_kv, D, R).view(B, T, H_kv, D).transpose(1, 2)
    s = dict(case=case, table=table, pos=torch.tensor(pos, dtype=torch.int32, device="cuda"),
             new=torch.tensor(new, dtype=torch.int32, device="cuda"),
             K=rows.to(dt).contiguous(), V=_rand(g, B, H_kv, T, D).to(dt), q=_rand(g, B, H_q, T, D).to(dt),
             P=_basis(g, H_kv, D) if case["basis"] else None, rope=_rope_angles(max(pos) + T, case["rot_dim"]))
    s["q_out"] = torch.zeros_like(s["q"])
    shape = (n_pages, H_kv, page, D)
    s["lo"] = torch.zeros(n_pages, H_kv, page, case["d_lo"], dtype=dt, device="cuda") if case["d_lo"] else None
    if case["op"] == "append":
        s["Kp"], s["Vp"] = _rand(g, *shape).to(dt), _rand(g, *shape).to(dt)
    else:
        s["Kp"], s["ks"] = _quantised(_rand(g, *shape), case["block"])
        s["Vp"], s["vs"] = _quantised(_rand(g, *shape) * 0.5, case["block"])
    return s


def _quantised(x, block):
    """x [n_pages, H, page, D] as e4m3 codes and their scales [n_pages, H, page / block]."""
    n, H, page, D = x.shape
    y = x.view(n, H, page // block, block * D)
    s = _pow2_scale(y.abs().amax(-1))
    return (y / s[..., None]).view(n, H, page, D).to(_F8), s


def _prepare_attention(case, g):
    B, H_q, H_kv, D, page, block = (case[k] for k in ("B", "H_q", "H_kv", "D", "page", "block"))
    lens = _lens(case)
    table, n_pages = _tables(case, [(0, -(-n // page)) for n in lens], g)
    R = _basis(g, H_kv, D)
    Kp = torch.empty(n_pages, H_kv, page, D, dtype=_F8, device="cuda")
    Vp, ks = torch.empty_like(Kp), torch.empty(n_pages, H_kv, page // block, device="cuda")
    vs = torch.empty_like(ks)
    step = max(1, (1 << 26) // (H_kv * page * D))
    for a in range(0, n_pages, step):
        m = min(step, n_pages - a)
        k = _keys(g, m * page, H_kv, D, R).view(m, page, H_kv, D).transpose(1, 2).contiguous()
        Kp[a:a + m], ks[a:a + m] = _quantised(k, block)
        Vp[a:a + m], vs[a:a + m] = _quantised(_rand(g, m, H_kv, page, D), block)
    # queries along the keys' directions, so that some tokens stand out
    G = H_q // H_kv
    q = _keys(g, B * G, H_kv, D, R).view(B, G, H_kv, D).transpose(1, 2).reshape(B, H_q, D) * 4
    s = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), Kp=Kp, Vp=Vp, ks=ks, vs=vs)
    if case["op"] == "dense8":
        s["q"] = q.to(_DT[case["dt"]]).contiguous()
        return s
    # each query head's own k tokens, ascending, -1 behind the last (a short sequence has fewer)
    k = case["k"]
    idx = torch.empty(B, H_q, k, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        m = min(k, n)
        idx[b] = -1
        if m:
            idx[b, :, :m] = torch.rand(H_q, n, generator=g, device="cuda").topk(m).indices.sort(-1).values.to(torch.int32)
    s["q"], s["idx"] = q.contiguous(), idx
    return s


def prepare(case, seed):
    g = _gen(seed)
    return _prepare_append(case, g) if case["op"] in ("append", "append8") else _prepare_attention(case, g)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rope(x, cs, interleaved):
    """Rows x [..., D] fp32 turned by cos/sin rows cs [..., rot_dim]."""
    r = cs.shape[-1]
    c, s = cs[..., : r // 2], cs[..., r // 2:]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., : r // 2], x[..., r // 2:r]
        y[..., : r // 2], y[..., r // 2:r] = a * c - b * s, a * s + b * c
    return y


def _plain_new_rows(s):
    """The appended tokens' rotated queries and keys, their (sequence, token) pairs and cache places."""
    c = s["case"]
    T, page = c["T"], c["page"]
    t = torch.arange(T, device="cuda")
    live = t < s["new"].long()[:, None]
    j = s["pos"].long()[:, None] + t
    cs = s["rope"][j.clamp(max=s["rope"].shape[0] - 1)][:, None]
    K = _rope(s["K"].float(), cs, c["interleaved"])
    if s["P"] is not None:
        K = torch.matmul(K, s["P"])
    s["q_out"].copy_(torch.where(live[:, None, :, None], _rope(s["q"].float(), cs, c["interleaved"]).to(s["q"].dtype), s["q_out"]))
    b, t = live.nonzero(as_tuple=True)
    j = j[b, t]
    return K, b, t, s["table"].long()[b, j // page], j % page


def _plain_append(s):
    K, b, t, pg, slot = _plain_new_rows(s)
    dt = s["K"].dtype
    s["Kp"][pg, :, slot] = K[b, :, t].to(dt)
    s["Vp"][pg, :, slot] = s["V"][b, :, t]
    if s["lo"] is not None:
        s["lo"][pg, :, slot] = K[b, :, t, : s["lo"].shape[-1]].to(dt)


def _plain_store8(s, X, b, t, pg, slot, pages, scales):
    """The rows X[b, :, t] into 8-bit pages, with their blocks' new scales and older tokens."""
    c = s["case"]
    block, page = c["block"], c["page"]
    nb = page // block
    # largest new magnitude of every touched block (the others stay at -1)
    cell = pg * nb + slot // block
    rows = X[b, :, t]
    amax = torch.full((pages.shape[0] * nb, X.shape[1]), -1.0, device="cuda")
    amax.index_reduce_(0, cell, rows.abs().amax(-1), "amax")
    first = torch.full((pages.shape[0] * nb,), block, dtype=torch.long, device="cuda")
    first.index_reduce_(0, cell, slot % block, "amin")  # older tokens sit before the first new one
    touched = (first < block).nonzero().squeeze(1)
    old = scales.transpose(1, 2).reshape(-1, scales.shape[1])[touched]
    grown = _pow2_scale(amax[touched])
    new = torch.where(first[touched, None] > 0, torch.maximum(old, grown), grown)
    p, k = touched // nb, touched % nb
    at = k[:, None] * block + torch.arange(block, device="cuda")
    # older codes to the new scale (a block without older tokens, or one whose scale stays, keeps its bytes)
    codes = pages.view(torch.uint8)[p[:, None], :, at].view(_F8)
    again = (codes.float() * (old / new)[:, None, :, None]).to(_F8)
    keep = (torch.arange(block, device="cuda") < first[touched, None])[:, :, None, None] & (old < new)[:, None, :, None]
    pages.view(torch.uint8)[p[:, None], :, at] = torch.where(keep, again.view(torch.uint8), codes.view(torch.uint8))
    scales[p, :, k] = new
    code = (rows / scales[pg, :, slot // block][..., None]).to(_F8)
    pages.view(torch.uint8)[pg, :, slot] = code.view(torch.uint8)


def _plain_append8(s):
    K, b, t, pg, slot = _plain_new_rows(s)
    if s["lo"] is not None:
        s["lo"][pg, :, slot] = K[b, :, t, : s["lo"].shape[-1]].to(s["K"].dtype)
    _plain_store8(s, K, b, t, pg, slot, s["Kp"], s["ks"])
    _plain_store8(s, s["V"].float(), b, t, pg, slot, s["Vp"], s["vs"])


def _plain_dense8(s):
    c = s["case"]
    B, H_kv, D, page, block, S = (c[k] for k in ("B", "H_kv", "D", "page", "block", "S"))
    G = c["H_q"] // H_kv
    pages = s["table"].long().clamp(min=0)
    n = pages.shape[1] * page
    live = torch.arange(n, device="cuda") < s["lens"].long()[:, None]

    def rows(codes, scales):
        x = codes.view(torch.uint8)[pages].view(_F8).float().view(B, -1, H_kv, page // block, block, D)
        x = x * scales[pages][..., None, None]
        x = x.view(B, -1, H_kv, page, D).transpose(1, 2).reshape(B, H_kv, n, D)
        return torch.where(live[:, None, :, None], x, torch.zeros((), device="cuda"))

    a = torch.matmul(s["q"].float().view(B, H_kv, G, D), rows(s["Kp"], s["ks"]).transpose(-1, -2)) / math.sqrt(D)
    a = a.masked_fill(~live[:, None, None], -math.inf)
    p = torch.exp(a - a.amax(-1, keepdim=True).clamp(min=-1e38))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows(s["Vp"], s["vs"])) / torch.where(l > 0, l, torch.ones_like(l))
    return o.view(B, H_kv * G, D).to(s["q"].dtype)


def _plain_sparse8(s):
    c = s["case"]
    B, H_q, H_kv, D, page, block = (c[k] for k in ("B", "H_q", "H_kv", "D", "page", "block"))
    idx = s["idx"].long()
    live = (idx >= 0) & (idx < s["lens"].long()[:, None, None])
    j = idx.clamp(min=0)
    pg = torch.gather(s["table"].long()[:, None].expand(B, H_q, -1), 2, j // page).clamp(min=0)
    row = (pg * H_kv + (torch.arange(H_q, device="cuda") // (H_q // H_kv))[:, None]) * page + j % page

    def rows(codes, scales):
        x = codes.view(torch.uint8).view(-1, D)[row].view(_F8).float() * scales.reshape(-1)[row // block][..., None]
        return torch.where(live[..., None], x, torch.zeros((), device="cuda"))

    a = torch.matmul(rows(s["Kp"], s["ks"]), s["q"][..., None]).squeeze(-1) / math.sqrt(D)
    a = a.masked_fill(~live, -math.inf)
    p = torch.exp(a - a.amax(-1, keepdim=True).clamp(min=-1e38))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p[:, :, None], rows(s["Vp"], s["vs"])).squeeze(2) / torch.where(l > 0, l, torch.ones_like(l))
    return o.to(_DT[c["dt"]])


def _outputs(s):
    op = s["case"]["op"]
    got = {"K": s["Kp"], "V": s["Vp"], "q": s["q_out"]}
    if s["lo"] is not None:
        got["plane"] = s["lo"]
    if op == "append8":
        got["k_scales"], got["v_scales"] = s["ks"], s["vs"]
    return got


def run(state):
    c = state["case"]
    s, op = state, c["op"]
    if own:
        m = _lib()
        if op == "append":
            m.loki_append_keys_paged_rope(s["K"], s["V"], s["P"], s["Kp"], s["Vp"], s["table"], s["pos"],
                                          rope_table=s["rope"], interleaved=c["interleaved"], Kt_lo_pages=s["lo"],
                                          new_lens=s["new"], q=s["q"], q_out=s["q_out"])
            return _outputs(s)
        if op == "append8":
            m.loki_append_keys_paged_q8(s["K"], s["V"], s["P"], s["Kp"], s["Vp"], s["ks"], s["vs"], s["table"],
                                        s["pos"], rope_table=s["rope"], interleaved=c["interleaved"],
                                        Kt_lo_pages=s["lo"], new_lens=s["new"], q=s["q"], q_out=s["q_out"])
            return _outputs(s)
        if op == "dense8":
            return m.dense_decode_attention_paged_q8(s["q"], s["Kp"], s["Vp"], s["ks"], s["vs"], s["table"], s["lens"])
        return m.loki_sparse_attention_paged_q8(s["q"], s["Kp"], s["Vp"], s["ks"], s["vs"], s["table"], s["lens"],
                                                s["idx"], dtype=_DT[c["dt"]])
    if op == "append":
        _plain_append(s)
        return _outputs(s)
    if op == "append8":
        _plain_append8(s)
        return _outputs(s)
    return _plain_dense8(s) if op == "dense8" else _plain_sparse8(s)


def work(case):
    """Each input read once and each output written once."""
    H_q, H_kv, D = case["H_q"], case["H_kv"], case["D"]
    e, n = _SIZE[case["dt"]], sum(_lens(case))
    if case["op"] in ("append", "append8"):
        out = (1 if case["op"] == "append8" else e) * 2 * D + e * case["d_lo"]
        spots = {p + t for p, m in zip(_positions(case), _lens(case)) for t in range(m)}
        by = n * H_kv * (2 * D * e + out) + n * H_q * D * 2 * e + len(spots) * case["rot_dim"] * 4
        by += 4 * H_kv * D * D if case["basis"] else 0
        if case["op"] == "append8":
            by += 8 * H_kv * sum(-(-m // case["block"]) for m in _lens(case))
        return {"bytes": by, "flops": n * H_kv * 2 * D * D * bool(case["basis"]) + 3 * n * (H_q + H_kv) * case["rot_dim"]}
    if case["op"] == "dense8":
        by = n * H_kv * 2 * D + 8 * H_kv * sum(-(-m // case["block"]) for m in _lens(case))
        return {"bytes": by + 2 * case["B"] * H_q * D * e, "flops": 4 * D * H_q * n}
    sel = H_q * sum(min(case["k"], m) for m in _lens(case))
    return {"bytes": sel * (2 * D + 8) + case["B"] * H_q * (4 * case["k"] + D * (4 + e)), "flops": 4 * D * sel}


# ---------------------------------------------------------------------------
# 64 bits, from the definition, sequence by sequence
# ---------------------------------------------------------------------------

def _exact_turn(x, case, j):
    """x [..., n, D] at positions j [n] with angles in 64 bits."""
    r = case["rot_dim"]
    i = np.arange(r // 2)
    lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
    ang = torch.from_numpy(np.outer(np.asarray(j, np.float64), 10000.0 ** (-2.0 * i / r))).cuda()
    y = x.clone()
    y[..., lo] = x[..., lo] * ang.cos() - x[..., hi] * ang.sin()
    y[..., hi] = x[..., hi] * ang.cos() + x[..., lo] * ang.sin()
    return y


def _exact_scale(top):
    """2^e with the least whole e >= -126 such that top <= 448 * 2^e."""
    if top <= 0:
        return 2.0 ** -126
    e = max(-126, math.ceil(math.log2(top / 448.0)) - 2)
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _exact_append(case, s):
    page, eight = case["page"], case["op"] == "append8"
    table = s["table"].cpu().numpy()
    K, V, q = s["K"].double(), s["V"].double(), s["q_out"].double()
    Kp, Vp = s["Kp"].double(), s["Vp"].double()
    lo = None if s["lo"] is None else s["lo"].double()
    ks, vs = (s["ks"].double(), s["vs"].double()) if eight else (None, None)
    for b, (n, p0) in enumerate(zip(_lens(case), _positions(case))):
        if n == 0:
            continue
        j = np.arange(p0, p0 + n)
        q[b, :, :n] = _exact_turn(s["q"][b, :, :n].double(), case, j)
        rows = _exact_turn(K[b, :, :n], case, j)
        if s["P"] is not None:
            rows = torch.einsum("hnd,hdc->hnc", rows, s["P"].double())
        pg, at = torch.from_numpy(table[b, j // page]).long().cuda(), torch.from_numpy(j % page).cuda()
        if lo is not None:
            lo[pg, :, at] = rows[:, :, : case["d_lo"]].transpose(0, 1)
        if not eight:
            Kp[pg, :, at], Vp[pg, :, at] = rows.transpose(0, 1), V[b, :, :n].transpose(0, 1)
            continue
        block = case["block"]
        for x, codes, scales in ((rows, Kp, ks), (V[b, :, :n], Vp, vs)):
            starts = sorted({p0} | {t for t in range(p0, p0 + n) if t % block == 0})
            ends = starts[1:] + [p0 + n]
            tops = torch.stack([x[:, a - p0:z - p0].abs().amax((1, 2)) for a, z in zip(starts, ends)]).cpu().numpy()
            sc = np.array([[_exact_scale(float(v)) for v in row] for row in tops])
            was = scales[table[b, p0 // page], :, p0 % page // block].cpu().numpy()
            if p0 % block:  # the block's older tokens keep their values at the larger scale
                sc[0] = np.maximum(sc[0], was)
                a = p0 % page - p0 % block
                codes[table[b, p0 // page], :, a:p0 % page] *= torch.from_numpy(was / sc[0]).cuda()[:, None, None]
            sc = torch.from_numpy(sc).cuda()
            which = torch.from_numpy(np.searchsorted(np.array(starts), j, side="right") - 1).cuda()
            codes[pg, :, at] = (x / sc[which].t()[:, :, None]).transpose(0, 1)
            for i, a in enumerate(starts):
                scales[table[b, a // page], :, a % page // block] = sc[i]
    got = {"K": Kp, "V": Vp, "q": q}
    if lo is not None:
        got["plane"] = lo
    if eight:
        got["k_scales"], got["v_scales"] = ks, vs
    return got


def _exact_attention(case, s):
    B, H_q, H_kv, D, page, block = (case[k] for k in ("B", "H_q", "H_kv", "D", "page", "block"))
    G = H_q // H_kv
    out = torch.zeros(B, H_q, D, dtype=torch.float64, device="cuda")
    ks, vs = s["ks"].double(), s["vs"].double()
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        pg, at = s["table"][b].long()[j // page], j % page
        for h in range(H_kv):
            K = s["Kp"].view(torch.uint8)[pg, h, at].view(_F8).double() * ks[pg, h, at // block][:, None]
            V = s["Vp"].view(torch.uint8)[pg, h, at].view(_F8).double() * vs[pg, h, at // block][:, None]
            a = s["q"][b, h * G:(h + 1) * G].double() @ K.t() / math.sqrt(D)
            if case["op"] == "sparse8":
                m = min(case["k"], n)
                chosen = torch.zeros(G, n, dtype=torch.bool, device="cuda")
                chosen.scatter_(1, s["idx"][b, h * G:(h + 1) * G, :m].long(), True)
                a = torch.where(chosen, a, torch.full_like(a, -math.inf))
            out[b, h * G:(h + 1) * G] = torch.softmax(a, -1) @ V
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] in ("append", "append8") else _exact_attention(case, s)
