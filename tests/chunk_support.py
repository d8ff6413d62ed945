"""References of the chunk operators in plain Python and float64 (test infrastructure only)."""

from __future__ import annotations

import numpy as np
import torch


def ceil_div(a, b):
    return -(-a // b)


def plan_reference(table, lens, delta, free, p: int, tokens: int) -> dict:
    """One plan step, request by request: ``table`` [B][width], ``lens`` and ``delta`` lists, ``free``
    the stack (last entry on top)."""
    table = np.array(table, copy=True)
    B, width = table.shape
    lens, stack = list(lens), list(free)
    want = [max(d, 0) for d in delta]
    start = [sum(want[:b]) for b in range(B + 1)]
    count = [0] * B
    refused = False
    for b in range(B):  # what is dropped goes back first
        if delta[b] < 0:
            keep_len = max(0, lens[b] + delta[b])
            for j in range(ceil_div(keep_len, p), ceil_div(lens[b], p)):
                stack.append(int(table[b, j]))
            lens[b] = keep_len
    wanted_so_far, top = 0, len(stack)
    new_lens = list(lens)
    for b in range(B):
        if want[b] == 0:
            continue
        n = lens[b] + want[b]
        if start[b + 1] > tokens or n > p * width:
            refused = True
            continue
        need = ceil_div(n, p) - ceil_div(lens[b], p)
        wanted_so_far += need
        if need and wanted_so_far > top:
            refused = True
            continue
        for j in range(ceil_div(lens[b], p), ceil_div(n, p)):
            table[b, j] = stack.pop()
        count[b], new_lens[b] = want[b], n
    row, pos, slot = [-1] * tokens, [-1] * tokens, [-1] * tokens
    for b in range(B):
        for i in range(count[b]):
            s = lens[b] + i
            row[start[b] + i], pos[start[b] + i] = b, s
            slot[start[b] + i] = int(table[b, s // p]) * p + s % p
    return dict(table=table, lens=new_lens, stack=stack, start=start, count=count, row=row, pos=pos,
                slot=slot, refused=refused)


def rotate_reference(x, positions, axis, inv_freq, interleaved: bool) -> np.ndarray:
    """float64 rotation of ``x`` [T][heads][D] by ``positions`` [axes][T]."""
    x = x.double().cpu().numpy().copy()
    pos = positions.cpu().numpy().astype(np.float64)
    half = len(inv_freq)
    for i in range(half):
        ang = pos[axis[i]] * inv_freq[i]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        xa, xb = x[..., a].copy(), x[..., b].copy()
        x[..., a], x[..., b] = xa * c - xb * s, xb * c + xa * s
    return x


def visible(pos, L: int, window) -> np.ndarray:
    """bool [n][L]: what the queries at positions ``pos`` see; ``window`` None or (sink, local)."""
    t = np.arange(L)[None, :]
    s = np.asarray(pos)[:, None]
    ok = t <= s
    if window is not None:
        sink, local = window
        ok &= (t < sink) | (t > s - local)
    return ok


def attend_reference(q, K, V, ok, scale: float):
    """float64 attention of rows ``q`` [R][D] over ``K``, ``V`` [L][D] where ``ok`` [R][L]:
    (O, m, l, A, d) with A = sum p |v| / l, the weight that a rounding of the probabilities moves, and
    d the largest error of a logit summed in fp32 (128 products, each rounded and added once)."""
    S = np.where(ok, scale * (q @ K.T), -np.inf)
    m = S.max(1, initial=-np.inf)
    P = np.exp(S - np.where(np.isneginf(m), 0.0, m)[:, None])
    l = P.sum(1)
    live = np.where(l > 0, l, 1.0)[:, None]
    Vz = np.where(ok.any(0)[:, None], V, 0.0)
    d = scale * 128 * 2.0 ** -24 * (np.abs(q) @ np.abs(np.where(ok.any(0)[:, None], K, 0.0)).T).max(
        initial=0.0)
    return P @ Vz / live, m, l, P @ np.abs(Vz) / live, d


def check_rows(got, ref, what: str):
    """(out bf16, m, l) rows against ``attend_reference``.  out: the stored value is rounded by at most
    2^-8 of itself, every probability by 2^-8 of itself before the product (which moves the sum by at
    most 2^-8 A), and a logit error d moves a probability and the sum by 2 d of themselves at most;
    2^-18 of A covers the fp32 sums and exponentials."""
    O, m, l, A, d = ref
    out, gm, gl = (t.double().cpu().numpy() for t in got)
    tol = 2.0 ** -8 * np.abs(O) * (1 + 2.0 ** -7) + (2.0 ** -8 + 4 * d + 2.0 ** -18) * A + 1e-30
    err = np.abs(out - O)
    assert (err <= tol).all(), f"{what} O: worst {np.max(err / tol):.2f} of its tolerance"
    inf = np.isneginf(m)
    assert (np.isneginf(gm) == inf).all(), f"{what} m: empty rows"
    assert (np.abs(np.where(inf, 0, gm) - np.where(inf, 0, m)) <= d + 2.0 ** -20 *
            np.abs(np.where(inf, 0, m))).all(), f"{what} m"
    assert (np.abs(gl - l) <= (4 * d + 2.0 ** -18) * l).all(), f"{what} l"


class ChunkCase:
    """Random pools and tables for requests of ``(tokens before, new tokens)``; every slot of the pool
    that no live token owns holds NaN."""

    def __init__(self, spec, page: int, hq: int, hkv: int, seed: int = 0, extra_tokens: int = 0,
                 streaming=None, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.spec, self.page, self.hq, self.hkv = spec, page, hq, hkv
        lens = [o + n for o, n in spec]
        used = [ceil_div(n, page) for n in lens]
        self.phys = sum(used) + 3
        width = max(used + [1]) + 1
        perm = torch.randperm(self.phys, generator=g).tolist()
        table = torch.full((len(spec), width), -1, dtype=torch.int32)
        k = torch.full((self.phys, hkv, page, 128), float("nan"))
        v = k.clone()
        for b, n in enumerate(lens):
            for j in range(used[b]):
                ph = perm.pop()
                table[b, j] = ph
                c = min(page, n - j * page)
                k[ph, :, :c] = torch.randn(hkv, c, 128, generator=g)
                v[ph, :, :c] = torch.randn(hkv, c, 128, generator=g)
        self.tokens = sum(n for _, n in spec) + extra_tokens
        start = np.concatenate([[0], np.cumsum([n for _, n in spec])]).astype(np.int32)
        q = torch.randn(self.tokens, hq, 128, generator=g)
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=device)
        self.k, self.v = k.bfloat16().to(device), v.bfloat16().to(device)
        self.table, self.lens, self.start = table.to(device), i32(lens), i32(start)
        self.count = i32([n for _, n in spec])
        self.q = q.bfloat16().to(device)
        self.streaming = None if streaming is None else torch.tensor(
            streaming, dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def rows(self, pool, b: int, h: int) -> np.ndarray:
        L = sum(self.spec[b])
        pages = self.table[b, :ceil_div(L, self.page)].long()
        return pool[pages, h].reshape(-1, 128)[:L].double().cpu().numpy()

    def check(self, out, m, l, scale: float, window=(0, 0), requests=None):
        """Compares every live row with the reference."""
        G = self.hq // self.hkv
        hs = [0] * self.hkv if self.streaming is None else self.streaming.cpu().tolist()
        for b, (o, n) in enumerate(self.spec):
            if n == 0 or (requests is not None and b not in requests):
                continue
            t0 = int(self.start[b])
            ok = {w: visible(np.arange(o, o + n), o + n, window if w else None) for w in (0, 1)}
            for h in range(self.hkv):
                K, V = self.rows(self.k, b, h), self.rows(self.v, b, h)
                for hh in range(h * G, (h + 1) * G):
                    ref = attend_reference(self.q[t0:t0 + n, hh].double().cpu().numpy(), K, V,
                                           ok[1 if hs[h] else 0], scale)
                    check_rows((out[t0:t0 + n, hh], m[t0:t0 + n, hh], l[t0:t0 + n, hh]), ref,
                               f"request {b} head {hh}")
