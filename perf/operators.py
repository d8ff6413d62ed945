"""Measured cases of the operators that bring a chunk of new tokens into the paged cache and attend it.

Four operators, each with a plain form in elementary torch operations and the library's own calls:

* ``plan``    block tables, slot maps and the page stack of a step, from request lengths
* ``append``  rotary positions of q and k, K and V into their pages, metadata of the touched pages
* ``attend``  causal attention of a ragged chunk over the paged cache (dense heads)
* ``window``  the same for streaming heads: the first ``sink`` tokens and the last ``local`` ones

Head counts, page sizes and context lengths are those of this repository's workloads (32 query heads
on 8, 2 or 32 KV heads, pages of 16 and 64 tokens, 4K to 128K tokens, 64 sink and 256 local tokens).
"""

from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

D = 128
ROPE_BASE = 500000.0


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # every request of a decode batch takes one more token: the call of every serving step
        dict(name="plan_decode", op="plan", batch=8, page=64, old_min=100000, old_max=131000,
             new_min=1, new_max=1, single=1.0, drop=0.0, lens=1),
        # a mixed step: decode, prompt chunks, finished or rolled-back requests
        dict(name="plan_mixed", op="plan", batch=256, page=16, old_min=1, old_max=8192,
             new_min=2, new_max=257, single=0.6, drop=0.1, lens=2),
        # thousands of requests with prompts of any length (offline batch)
        dict(name="plan_large", op="plan", batch=2048, page=16, old_min=1, old_max=4096,
             new_min=1, new_max=127, single=0.3, drop=0.05, lens=3),
        # decode step of the llama layer: one token per request, min/max metadata
        dict(name="append_decode", op="append", batch=4, q_heads=32, kv_heads=8, page=16,
             old_min=32000, old_max=32700, new_min=1, new_max=1, single=1.0, kind="minmax",
             logical=16, axes=1, rot=128, interleaved=False, lens=4),
        # a ragged prompt batch with time/height/width positions, hierarchical pages
        dict(name="append_axes", op="append", batch=6, q_heads=32, kv_heads=8, page=64,
             old_min=0, old_max=4096, new_min=700, new_max=2049, single=0.0, kind="minmax",
             logical=16, axes=3, rot=128, interleaved=False, lens=5),
        # MHA with mean-key blocks, partly rotated heads, neighbouring pairs
        dict(name="append_mean", op="append", batch=4, q_heads=32, kv_heads=32, page=16,
             old_min=1, old_max=2000, new_min=900, new_max=1100, single=0.0, kind="mean",
             logical=16, axes=1, rot=64, interleaved=True, lens=6),
        # dense decode of the llama layer: one token per request over 32K
        dict(name="attend_decode", op="attend", batch=4, q_heads=32, kv_heads=8, page=16,
             old_min=32000, old_max=32760, new_min=1, new_max=1, single=1.0, lens=7),
        # a prompt's next chunk over a long context
        dict(name="attend_chunk", op="attend", batch=1, q_heads=32, kv_heads=8, page=16,
             old_min=30000, old_max=30720, new_min=2048, new_max=2048, single=0.0, lens=8),
        # decode requests and prompt chunks in one step, 16 query heads on a KV head
        dict(name="attend_mixed", op="attend", batch=7, q_heads=32, kv_heads=2, page=64,
             old_min=200, old_max=12000, new_min=60, new_max=700, single=0.5, lens=9),
        # whole prompts of an MHA model
        dict(name="attend_prompt", op="attend", batch=1, q_heads=32, kv_heads=32, page=16,
             old_min=0, old_max=0, new_min=8191, new_max=8191, single=0.0, lens=10),
        # streaming heads of a decode batch at 128K
        dict(name="window_decode", op="window", batch=8, q_heads=32, kv_heads=8, page=64,
             old_min=120000, old_max=131000, new_min=1, new_max=1, single=1.0, sink=64, local=256,
             lens=11),
        # streaming heads of a long prompt
        dict(name="window_prompt", op="window", batch=2, q_heads=32, kv_heads=8, page=64,
             old_min=1, old_max=3000, new_min=4000, new_max=6000, single=0.0, sink=64, local=1000,
             lens=12),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "window"])
    c = dict(op=op, page=rng.choice([16, 16, 32, 48, 64, 128]), lens=rng.randrange(1 << 20))
    single = rng.choice([0.0, 0.3, 0.7, 1.0])
    if op == "plan":
        n = _logint(rng, 1, 300)
        return dict(c, batch=_logint(rng, 1, 1500), old_min=1, old_max=_logint(rng, 100, 8000),
                    new_min=1, new_max=n, single=single, drop=rng.choice([0.0, 0.1, 0.3]))
    heads = rng.choice([(32, 8), (32, 2), (32, 32), (4, 1), (24, 8), (28, 4), (40, 8)])
    c = dict(c, q_heads=heads[0], kv_heads=heads[1], single=single)
    n = _logint(rng, 1, 1500)
    if op == "append":
        kind = rng.choice(["minmax", "mean"])
        return dict(c, batch=_logint(rng, 1, 8), old_min=0, old_max=_logint(rng, 10, 6000),
                    new_min=max(1, n // 3), new_max=n, kind=kind,
                    logical=rng.choice([16, c["page"]]), axes=rng.choice([1, 1, 2, 3]),
                    rot=rng.choice([32, 64, 96, 128]), interleaved=rng.random() < 0.4)
    batch = _logint(rng, 1, 6)
    old = _logint(rng, 100, 20000)
    # the padded score matrix of the plain form bounds what a case may hold
    while batch * n * (old + n) * heads[0] > 1.2e9:
        old, n = max(1, old * 2 // 3), max(1, n * 4 // 5)
    c = dict(c, batch=batch, old_min=0, old_max=old, new_min=max(1, n // 4), new_max=n)
    if op == "window":
        c = dict(c, sink=rng.choice([0, 4, 64, 128]), local=_logint(rng, 1, 2000))
    return c


def _lens(c):
    """(tokens before, change) of every request; the change is negative where tokens are dropped."""
    r = random.Random(c["lens"])
    old, new = [], []
    for _ in range(c["batch"]):
        o = r.randint(c["old_min"], c["old_max"])
        n = 1 if r.random() < c["single"] else r.randint(c["new_min"], c["new_max"])
        if c["op"] == "plan" and r.random() < c["drop"]:
            n = -o if r.random() < 0.5 else -min(o, r.randint(1, 40))
        old.append(o)
        new.append(n)
    return old, new


def _ceil(a, b):
    return -(-a // b)


def work(case):
    c = case
    old, new = _lens(c)
    B, p = c["batch"], c["page"]
    T = sum(max(n, 0) for n in new)
    if c["op"] == "plan":
        moved = sum(abs(_ceil(o + n, p) - _ceil(o, p)) for o, n in zip(old, new))
        return dict(bytes=B * 4 * 5 + T * 12 + moved * 8, flops=T + B)
    Hq, Hkv = c["q_heads"], c["kv_heads"]
    if c["op"] == "append":
        g = p // c["logical"]
        pages = sum(_ceil(o + n, p) - o // p for o, n in zip(old, new))
        held = sum(o % p for o in old)  # older keys of a partly filled first page
        return dict(bytes=2 * T * Hq * D * 2 + 4 * T * Hkv * D * 2 + held * Hkv * D * 2 +
                    pages * Hkv * g * D * 4, flops=6 * T * (Hq + Hkv) * c["rot"] // 2)
    pairs = live = 0
    for o, n in zip(old, new):
        pos = np.arange(o, o + n, dtype=np.int64)
        if c["op"] == "attend":
            pairs += int((pos + 1).sum())
            live += o + n
        else:
            pairs += int(np.minimum(pos + 1, np.minimum(c["sink"], np.maximum(
                pos + 1 - c["local"], 0)) + c["local"]).sum())
            first = max(0, o + 1 - c["local"])
            live += min(c["sink"], first) + (o + n - first)
    return dict(bytes=2 * T * Hq * D * 2 + T * Hq * 8 + live * Hkv * D * 4, flops=4 * D * Hq * pairs)


# ---------------------------------------------------------------------------------------- prepare

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _rope_axes(c):
    """Axis of every rotated pair: contiguous sections, the first the longest."""
    half = c["rot"] // 2
    cut = [half * (i + 1) // c["axes"] for i in range(c["axes"])]
    return [next(a for a, e in enumerate(cut) if i < e) for i in range(half)]


def _positions(c, old, new, rng):
    """int32 [axes][T]: one axis counts tokens; of several, the first counts frames of 8 x 12 patches."""
    rows = []
    for o, n in zip(old, new):
        t = np.arange(o, o + n)
        off = rng.randrange(0, 1 << 18)  # a long conversation before this prompt
        rows.append(np.stack([t + off] if c["axes"] == 1 else
                             [off + t // 96, off + t // 12 % 8, off + t % 12][:c["axes"]]))
    return _i32(np.concatenate(rows, axis=1))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = random.Random(seed)
    old, new = _lens(c)
    B, p = c["batch"], c["page"]
    most = max(_ceil(o + max(n, 0), p) for o, n in zip(old, new)) + 1
    held = sum(_ceil(o, p) for o in old)
    if c["op"] == "plan":
        need = sum(max(0, _ceil(o + n, p) - _ceil(o, p)) for o, n in zip(old, new) if n > 0)
        phys = held + need + 7
        perm = torch.randperm(phys, generator=g, device="cuda").to(torch.int32)
        cnt = torch.tensor([_ceil(o, p) for o in old], device="cuda")
        first = torch.cumsum(cnt, 0) - cnt
        j = torch.arange(most, device="cuda")
        table = torch.where(j < cnt[:, None], perm[(first[:, None] + j).clamp(max=phys - 1)],
                            torch.full((), -1, dtype=torch.int32, device="cuda"))
        free = torch.full((phys,), -1, dtype=torch.int32, device="cuda")
        free[:phys - held] = perm[held:]
        return dict(case=c, table=table.contiguous(), old=_i32(old), delta=_i32(new), free=free,
                    free_in=_i32([phys - held]), tokens=sum(max(n, 0) for n in new), phys=phys)
    Hq, Hkv = c["q_heads"], c["kv_heads"]
    T = sum(new)
    # every page of a request is assigned already; a few pages of the pool belong to nobody
    lens = [o + n for o, n in zip(old, new)]
    cnt = torch.tensor([_ceil(n, p) for n in lens], device="cuda")
    phys = int(cnt.sum()) + 3
    perm = torch.randperm(phys, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(cnt, 0) - cnt
    j = torch.arange(most, device="cuda")
    table = torch.where(j < cnt[:, None], perm[(first[:, None] + j).clamp(max=phys - 1)],
                        torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()
    start = np.concatenate([[0], np.cumsum(new)])
    row = np.repeat(np.arange(B), new)
    pos = np.concatenate([np.arange(o, o + n) for o, n in zip(old, new)])
    s = dict(case=c, table=table, lens=_i32(lens), start=_i32(start), count=_i32(new), row=_i32(row),
             pos=_i32(pos), k_pages=_normal(g, phys, Hkv, p, D), v_pages=_normal(g, phys, Hkv, p, D),
             q=_normal(g, T, Hq, D), longest=max(lens), most_new=max(new))
    if c["op"] == "append":
        s.update(k=_normal(g, T, Hkv, D), v=_normal(g, T, Hkv, D), axis=_rope_axes(c),
                 positions=_positions(c, old, new, rng),
                 inv_freq=[ROPE_BASE ** (-2 * i / c["rot"]) for i in range(c["rot"] // 2)])
        n_sub = p // c["logical"]
        s["meta"] = (torch.zeros(phys, Hkv, n_sub, D, 2, dtype=torch.bfloat16, device="cuda")
                     if c["kind"] == "minmax" else
                     torch.zeros(phys, Hkv, n_sub, D, dtype=torch.float32, device="cuda"))
    elif c["op"] == "window":
        s["streaming"] = torch.ones(Hkv, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------ plain forms

def _plan_plain(s):
    p, T = s["case"]["page"], s["tokens"]
    L, d = s["old"].long(), s["delta"].long()
    B, width = s["table"].shape
    new = torch.clamp(d, min=0)
    start = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    kept = torch.clamp(L + torch.clamp(d, max=0), min=0)
    have, keep = (L + p - 1) // p, (kept + p - 1) // p
    gone = have - keep
    gone_end = torch.cumsum(gone, 0)
    F = s["free_in"].long()
    top = F + gone_end[-1]
    fits = (start[1:] <= T) & (L + new <= p * width)
    need = torch.where(fits & (new > 0), (L + new + p - 1) // p - have, torch.zeros_like(L))
    need_end = torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (need_end <= top))  # who needs no page is never held up
    need = torch.where(ok, need, torch.zeros_like(need))
    count = torch.where(ok, new, torch.zeros_like(new))
    lens = torch.where(d < 0, kept, L + count)
    # pages given back, in request and position order, on top of the stack
    total_gone, total_need = s["phys"], s["phys"]
    i = torch.arange(total_gone, device="cuda")
    b = torch.clamp(torch.searchsorted(gone_end, i, right=True), max=B - 1)
    j = torch.clamp(keep[b] + i - (gone_end - gone)[b], 0, width - 1)
    live = i < gone_end[-1]
    cap = s["free"].shape[0]
    stack = torch.cat([s["free"], torch.zeros(cap + 1, dtype=torch.int32, device="cuda")])
    at = torch.where(live, F + i, torch.full_like(i, 2 * cap))
    stack[at] = torch.where(live, s["table"][b, j], torch.zeros((), dtype=torch.int32, device="cuda"))
    # pages taken from the top
    taken_end = torch.cumsum(need, 0)
    i = torch.arange(total_need, device="cuda")
    b = torch.clamp(torch.searchsorted(taken_end, i, right=True), max=B - 1)
    j = have[b] + i - (taken_end - need)[b]
    live = i < taken_end[-1]
    page = stack[torch.clamp(top - 1 - i, min=0)]
    table = torch.cat([s["table"].reshape(-1), s["table"].new_zeros(1)])
    table[torch.where(live, b * width + j, torch.full_like(i, B * width))] = page
    table = table[:-1].reshape(B, width)
    left = top - taken_end[-1]
    k = torch.arange(cap, device="cuda")
    free = torch.where((k >= F) & (k < left), stack[:cap], s["free"])
    # the tokens
    t = torch.arange(T, device="cuda")
    b = torch.clamp(torch.searchsorted(start[1:], t, right=True), max=B - 1)
    live = (t < start[-1]) & (count[b] > 0)
    pos = L[b] + t - start[b]
    slot = table[b, torch.clamp(pos // p, 0, width - 1)].long() * p + pos % p
    none = torch.full_like(t, -1)
    i32 = torch.int32
    return dict(start=start.to(i32), count=count.to(i32), row=torch.where(live, b, none).to(i32),
                pos=torch.where(live, pos, none).to(i32), slot=torch.where(live, slot, none).to(i32),
                lens=lens.to(i32), table=table, free=free, left=left.to(i32))


def _rotate_plain(x, cos, sin, rot, interleaved):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2],
                                                                   x[..., rot // 2:rot])
    c, s = cos[:, None, :], sin[:, None, :]
    u, v = a * c - b * s, b * c + a * s
    r = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([r, x[..., rot:]], -1).to(torch.bfloat16)


def _append_plain(s):
    c = s["case"]
    p, lp, rot = c["page"], c["logical"], c["rot"]
    freq = torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda")
    axis = torch.tensor(s["axis"], device="cuda")
    angle = s["positions"].double()[axis].T * freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotate_plain(s["q"], cos, sin, rot, c["interleaved"])
    k = _rotate_plain(s["k"], cos, sin, rot, c["interleaved"])
    row, pos = s["row"].long(), s["pos"].long()
    phys = s["table"][row, pos // p].long()
    s["k_pages"][phys, :, pos % p] = k
    s["v_pages"][phys, :, pos % p] = s["v"]
    # metadata of the pages that hold a new token: one entry per (request, page position)
    lens, count = s["lens"].long(), s["count"].long()
    j0 = (lens - count) // p
    j = j0[:, None] + torch.arange((s["most_new"] - 1) // p + 2, device="cuda")
    b, i = torch.nonzero((j * p < lens[:, None]) & (count > 0)[:, None], as_tuple=True)
    j = j[b, i]
    at = s["table"][b, j].long()
    keys = s["k_pages"][at].float()  # [n][Hkv][p][D]
    n, H = keys.shape[:2]
    keys = keys.view(n, H, p // lp, lp, D)
    valid = (torch.arange(p, device="cuda") + j[:, None] * p < lens[b][:, None]).view(n, 1, p // lp,
                                                                                  lp, 1)
    some = valid.any(3)
    if c["kind"] == "minmax":
        hi = keys.masked_fill(~valid, -math.inf).amax(3)
        lo = keys.masked_fill(~valid, math.inf).amin(3)
        m = torch.where(some[..., None], torch.stack([hi, lo], -1), torch.zeros_like(hi)[..., None])
        s["meta"][at] = m.to(torch.bfloat16)
    else:
        total = keys.masked_fill(~valid, 0.0).double().sum(3)
        s["meta"][at] = (total / valid.sum(3).clamp(min=1)).float()
    return dict(q=q, k_pages=s["k_pages"], v_pages=s["v_pages"], meta=s["meta"])


def _attend_plain(s):
    c = s["case"]
    p, Hq, Hkv = c["page"], c["q_heads"], c["kv_heads"]
    B, G, N, Lm = c["batch"], Hq // Hkv, s["most_new"], s["longest"]
    lens, count, start = s["lens"].long(), s["count"].long(), s["start"].long()
    T = s["q"].shape[0]
    i = torch.arange(N, device="cuda")
    at = torch.where(i < count[:, None], start[:B, None] + i, torch.zeros_like(i))  # [B][N]
    pos = (lens - count)[:, None] + i
    t = torch.arange(Lm, device="cuda")
    phys = torch.clamp(s["table"][:, t // p].long(), min=0)  # [B][L]
    K = s["k_pages"][phys, :, t % p].float().permute(0, 2, 3, 1)  # [B][Hkv][D][L]
    V = s["v_pages"][phys, :, t % p].float().permute(0, 2, 1, 3)  # [B][Hkv][L][D]
    V = V.masked_fill((t >= lens[:, None])[:, None, :, None], 0.0)
    Q = s["q"][at].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    S = torch.matmul(Q, K).mul_(1.0 / math.sqrt(D)).view(B, Hkv, N, G, Lm)
    seen = (t <= pos[..., None]) & (i < count[:, None])[..., None]  # [B][N][L]
    if c["op"] == "window":
        seen &= (t < c["sink"]) | (t > pos[..., None] - c["local"])
    S.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = S.amax(-1)
    P = S.sub_(torch.where(m > -math.inf, m, torch.zeros_like(m))[..., None]).exp_()
    l = P.sum(-1)
    O = torch.matmul(P.view(B, Hkv, N * G, Lm), V).view(B, Hkv, N, G, D)
    O = torch.where(l[..., None] > 0, O / l[..., None], torch.zeros_like(O))
    b, i = torch.nonzero(i < count[:, None], as_tuple=True)  # in token order
    out = O[b, :, i].reshape(T, Hq, D).to(torch.bfloat16)
    return dict(out=out, m=m[b, :, i].reshape(T, Hq), l=l[b, :, i].reshape(T, Hq))


# --------------------------------------------------------------------------- the library's own calls

def _handle(s):
    """Descriptors, workspaces and output buffers: what a program keeps next to its cache."""
    from dynamic_block_sparse_gb300 import binding as lib
    c = s["case"]
    h = s["handle"] = dict(lib=lib)
    status = h["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    B = c["batch"]
    if c["op"] == "plan":
        T = s["tokens"]
        i32 = dict(dtype=torch.int32, device="cuda")
        h["out"] = o = dict(start=torch.empty(B + 1, **i32), count=torch.empty(B, **i32),
                            row=torch.empty(T, **i32), pos=torch.empty(T, **i32),
                            slot=torch.empty(T, **i32), lens=torch.empty(B, **i32),
                            table=s["table"].clone(), free=s["free"].clone(),
                            left=torch.empty(1, **i32))
        h["tables"] = lib.page_tables(o["table"], o["lens"], c["page"], s["phys"], status)
        h["chunk"] = lib.chunk(o["start"], o["count"], o["row"], o["pos"], o["slot"])
        h["ws"] = torch.zeros(lib.dsa_plan_chunk_workspace_size(B), dtype=torch.uint8, device="cuda")
        return h
    h["kv"] = lib.paged_kv(s["k_pages"], s["v_pages"], s["table"], s["lens"], c["q_heads"],
                           s.get("streaming"), status)
    h["chunk"] = lib.chunk(s["start"], s["count"], s["row"], s["pos"])
    if c["op"] == "append":
        h["rotary"] = lib.rotary(lib.rotary_phases(s["inv_freq"], "cuda"), c["rot"],
                                 torch.tensor(s["axis"], dtype=torch.uint8, device="cuda"),
                                 s["positions"], c["interleaved"])
        h["q"] = torch.empty_like(s["q"])
        h["kind"] = lib.DSA_META_MINMAX if c["kind"] == "minmax" else lib.DSA_META_MEAN
        return h
    T, Hq = s["q"].shape[:2]
    h["out"] = dict(out=torch.empty_like(s["q"]),
                    m=torch.empty(T, Hq, dtype=torch.float32, device="cuda"),
                    l=torch.empty(T, Hq, dtype=torch.float32, device="cuda"))
    h["ws"] = torch.zeros(lib.dsa_chunk_attn_workspace_size(h["kv"], T), dtype=torch.uint8,
                          device="cuda")
    return h


def _own(s):
    c = s["case"]
    h = s.get("handle") or _handle(s)
    lib = h["lib"]
    if c["op"] == "plan":
        lib.dsa_plan_chunk(h["tables"], s["old"], s["delta"], h["out"]["free"], s["free_in"],
                           h["out"]["left"], h["chunk"], h["ws"])
        return h["out"]
    if c["op"] == "append":
        lib.dsa_append_chunk(h["kv"], h["chunk"], s["k"], s["v"], h["rotary"], s["q"], h["q"],
                             h["kind"], c["logical"], s["meta"])
        return dict(q=h["q"], k_pages=s["k_pages"], v_pages=s["v_pages"], meta=s["meta"])
    o = h["out"]
    lib.dsa_chunk_attn(h["kv"], h["chunk"], s["q"], 1.0 / math.sqrt(D), o["out"], o["m"], o["l"],
                       h["ws"], sink=c.get("sink", 0), local=c.get("local", 0))
    return o


def run(state):
    if own:
        return _own(state)
    return {"plan": _plan_plain, "append": _append_plain, "attend": _attend_plain,
            "window": _attend_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- definition, 64 bits

def _exact_append(s):
    c = s["case"]
    p, lp, rot = c["page"], c["logical"], c["rot"]
    half = rot // 2
    pos = s["positions"].cpu().numpy().astype(np.float64)
    ang = np.stack([pos[s["axis"][i]] * s["inv_freq"][i] for i in range(half)], 1)
    e = torch.from_numpy(np.exp(1j * ang)).cuda()[:, None, :]

    def turn(x):
        y = x.double().clone()
        i = torch.arange(half, device="cuda")
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        z = torch.complex(y[..., a], y[..., b]) * e
        y[..., a], y[..., b] = z.real.contiguous(), z.imag.contiguous()
        return y

    k = turn(s["k"])
    kp, vp, meta = s["k_pages"].double(), s["v_pages"].double(), s["meta"].double()
    table, start = s["table"].cpu().tolist(), s["start"].cpu().tolist()
    for b, (n, L) in enumerate(zip(s["count"].cpu().tolist(), s["lens"].cpu().tolist())):
        for j in range((L - n) // p, _ceil(L, p)):
            page, lo, hi = table[b][j], max(L - n, j * p), min(L, (j + 1) * p)
            src = slice(start[b] + lo - (L - n), start[b] + hi - (L - n))
            kp[page, :, lo - j * p:hi - j * p] = k[src].transpose(0, 1)
            vp[page, :, lo - j * p:hi - j * p] = s["v"][src].double().transpose(0, 1)
            for sub in range(p // lp):
                x = kp[page, :, sub * lp:min((sub + 1) * lp, hi - j * p)]
                if x.shape[1] == 0 or sub * lp >= hi - j * p:
                    meta[page, :, sub] = 0
                elif c["kind"] == "minmax":
                    meta[page, :, sub] = torch.stack([x.amax(1), x.amin(1)], -1)
                else:
                    # the mean is of the keys as the cache holds them
                    meta[page, :, sub] = x.to(torch.bfloat16).double().mean(1)
    return dict(q=turn(s["q"]), k_pages=kp, v_pages=vp, meta=meta)


def _exact_attend(s):
    c = s["case"]
    p, Hq, Hkv = c["page"], c["q_heads"], c["kv_heads"]
    G, T = Hq // Hkv, s["q"].shape[0]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    m = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    l = torch.zeros(T, Hq, dtype=torch.float64, device="cuda")
    for b, (n, L) in enumerate(zip(s["count"].cpu().tolist(), s["lens"].cpu().tolist())):
        pages = s["table"][b, :_ceil(L, p)].long()
        t0 = int(s["start"][b])
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        t = torch.arange(L, device="cuda")[None, :]
        hidden = t > pos
        if c["op"] == "window":
            hidden |= (t >= c["sink"]) & (t <= pos - c["local"])
        for h in range(Hkv):
            K = s["k_pages"][pages, h].reshape(-1, D)[:L].double()
            V = s["v_pages"][pages, h].reshape(-1, D)[:L].double()
            for head in range(h * G, (h + 1) * G):
                S = (s["q"][t0:t0 + n, head].double() @ K.T) / math.sqrt(D)
                S[hidden] = -math.inf
                top = S.amax(1)
                E = torch.exp(S - top.clamp(min=-1e300)[:, None])
                z = E.sum(1)
                m[t0:t0 + n, head], l[t0:t0 + n, head] = top, z
                out[t0:t0 + n, head] = (E @ V) / z.clamp(min=1e-300)[:, None]
    return dict(out=out, m=m, l=l)


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
