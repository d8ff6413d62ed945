"""GPU parity of the chunk operators: the page plan against a request-by-request reference, the rotary
append against float64 rotation and the metadata build, the chunk attention against float64 softmax
attention, each at the sizes and masks where it can go wrong."""

import math
import random

import numpy as np
import pytest
import torch

from chunk_support import ChunkCase, ceil_div, plan_reference, rotate_reference
from dynamic_block_sparse_gb300 import binding as B

pytestmark = pytest.mark.gpu
I32 = torch.int32
SCALE = 1 / math.sqrt(128)


def _t(x, dtype=I32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


# ---------------------------------------------------------------------------------------------- plan

class _Plan:
    def __init__(self, table, lens, free, p, tokens, cap=None):
        self.p, self.tokens = p, tokens
        self.table, self.lens = _t(table), _t(lens)
        nb = len(lens)
        stack = list(free) + [-9] * ((cap if cap is not None else len(free) + 64) - len(free))
        self.free, self.top = _t(stack), _t([len(free)])
        e = lambda n: torch.full((n,), -77, dtype=I32, device="cuda")
        self.start, self.count = e(nb + 1), e(nb)
        self.row, self.pos, self.slot = e(tokens), e(tokens), e(tokens)
        self.status = torch.zeros(1, dtype=I32, device="cuda")
        self.kv = B.page_tables(self.table, self.lens, p, 1 << 20, self.status)
        self.chunk = B.chunk(self.start, self.count, self.row, self.pos, self.slot)
        self.ws = torch.zeros(B.dsa_plan_chunk_workspace_size(nb), dtype=torch.uint8, device="cuda")

    def step(self, delta):
        B.dsa_plan_chunk(self.kv, self.lens, _t(delta), self.free, self.top, self.top, self.chunk,
                         self.ws)

    def check(self, ref):
        torch.cuda.synchronize()
        assert self.lens.tolist() == ref["lens"]
        assert self.start.tolist() == ref["start"] and self.count.tolist() == ref["count"]
        assert self.row.tolist() == ref["row"] and self.pos.tolist() == ref["pos"]
        assert self.slot.tolist() == ref["slot"]
        assert (self.table.cpu().numpy() == ref["table"]).all()
        n = int(self.top)
        assert n == len(ref["stack"]) and self.free[:n].tolist() == ref["stack"]
        assert int(self.status) == (B.DSA_STATUS_NO_PAGES if ref["refused"] else 0)
        assert not self.ws.any()


@pytest.mark.parametrize("batch,p,tokens,width", [
    (1, 16, 1, 1), (1, 64, 0, 4), (3, 48, 50, 9), (8, 16, 40, 6), (31, 32, 700, 20),
    (513, 16, 5000, 9), (1500, 16, 9000, 5), (8192, 16, 8192, 2)])
def test_plan_steps(batch, p, tokens, width):
    """Several steps of growth, rollback and release, in place; the stack runs short in some."""
    r = random.Random(batch * 7 + p)
    phys = max(3, batch * width // 2)
    table = np.full((batch, width), -7)
    lens, free = [0] * batch, r.sample(range(phys), phys)
    pl = _Plan(table, lens, free, p, tokens, cap=phys)
    for _ in range(5):
        per = max(1, tokens // batch)
        delta = [r.choice([0, 1, 1, r.randint(1, 2 * per), r.randint(1, p * width), -r.randint(1, 40),
                           -(1 << 31)]) if batch < 100 else
                 r.choice([0, 1, 1, 1, r.randint(1, 2 * per), -r.randint(1, 40), -(1 << 31)])
                 for _ in range(batch)]
        ref = plan_reference(table, lens, delta, free, p, tokens)
        pl.status.zero_()
        pl.step(delta)
        pl.check(ref)
        table, lens, free = ref["table"], ref["lens"], ref["stack"]


def test_plan_out_of_place_and_huge_requests():
    """Separate inputs stay as they were, a request beyond 2^31 tokens is refused, and a stack that is
    too small for what comes back loses the surplus and says so."""
    table = np.arange(8).reshape(2, 4)
    pl = _Plan(table, [30, 64], [8, 9], 16, 16, cap=3)
    lens_in, fin = _t([30, 64]), _t([2])
    fout = _t([-1])
    B.dsa_plan_chunk(pl.kv, lens_in, _t([3, -64]), pl.free, fin, fout, pl.chunk, pl.ws)
    torch.cuda.synchronize()
    assert lens_in.tolist() == [30, 64] and fin.item() == 2
    # pushed 4 5 6 7 on [8, 9]; request 0 (33 tokens) takes 7; 5 are left, the stack holds 3
    assert pl.lens.tolist() == [33, 0] and pl.table[0].tolist() == [0, 1, 7, 3]
    assert fout.item() == 3 and pl.free.tolist() == [8, 9, 4]
    assert int(pl.status) == B.DSA_STATUS_OVERFLOW
    pl = _Plan(table, [1, 1], [8, 9], 16, 16)
    pl.step([(1 << 31) - 1, (1 << 31) - 1])
    torch.cuda.synchronize()
    assert pl.count.tolist() == [0, 0] and pl.lens.tolist() == [1, 1]
    assert pl.start.tolist() == [0, (1 << 31) - 1, (1 << 31) - 1]  # saturated
    assert int(pl.status) == B.DSA_STATUS_NO_PAGES and (pl.row == -1).all()


def test_plan_bad_ids_raise_status():
    """A page id outside the pool (from the table or the stack) gives slot -1 and a status."""
    pl = _Plan([[5, -1], [3, -1]], [8, 16], [1 << 21], 16, 4)
    pl.table[0, 0] = -4
    pl.step([2, 1])
    torch.cuda.synchronize()
    assert pl.slot.tolist() == [-1, -1, -1, -1] and pl.row.tolist() == [0, 0, 1, -1]
    assert int(pl.status) == B.DSA_STATUS_BAD_PAGE


# -------------------------------------------------------------------------------------------- append

def _chunk_of(case, tokens=None):
    n = case.tokens if tokens is None else tokens
    row, pos = np.full(n, -1), np.full(n, -1)
    t = 0
    for b, (o, k) in enumerate(case.spec):
        row[t:t + k], pos[t:t + k] = b, np.arange(o, o + k)
        t += k
    return B.chunk(case.start, case.count, _t(row), _t(pos))


def _meta(case, kind, lp, fill=7.0):
    g = case.page // lp
    if kind == B.DSA_META_MINMAX:
        return torch.full((case.phys, case.hkv, g, 128, 2), fill, dtype=torch.bfloat16, device="cuda")
    return torch.full((case.phys, case.hkv, g, 128), fill, dtype=torch.float32, device="cuda")


APPEND = [
    # spec, page, hq, hkv, lp, kind, rot, axes, interleaved
    ([(0, 1)], 16, 4, 1, 16, 0, 128, 1, False),
    ([(37, 1), (0, 1), (63, 1), (64, 1), (5, 0)], 64, 8, 2, 16, 0, 128, 1, False),
    ([(0, 200), (13, 70), (0, 0), (95, 1)], 48, 6, 2, 16, 1, 64, 3, True),
    ([(130, 300), (256, 5)], 256, 5, 5, 8, 0, 96, 2, False),
    ([(3, 29), (16, 16), (15, 2)], 16, 16, 1, 4, 1, 32, 4, False),
    ([(100, 257)], 128, 9, 3, 64, 0, 16, 1, True),
    ([(1, 1000), (0, 13)], 32, 32, 8, 32, 1, 128, 1, True),
]


@pytest.mark.parametrize("case_", APPEND)
def test_append_chunk(case_):
    spec, page, hq, hkv, lp, kind, rot, axes, inter = case_
    c = ChunkCase(spec, page, hq, hkv, seed=3, extra_tokens=5)
    T = c.tokens
    chunk = _chunk_of(c)
    g = torch.Generator().manual_seed(9)
    fused = torch.randn(T, hq + 2 * hkv + 1, 128, generator=g).bfloat16().cuda()
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:hq + 2 * hkv]
    half = rot // 2
    freq = [500000.0 ** (-2 * i / rot) for i in range(half)]
    axis = [i * axes // half for i in range(half)]
    r = random.Random(5)
    positions = _t([[r.randrange(-50, 1 << 20) for _ in range(T)] for _ in range(axes)])
    rot_d = B.rotary(B.rotary_phases(freq), rot, _t(axis, torch.uint8), positions, inter)
    live = sum(n for _, n in spec)
    # metadata as it stood before the chunk, built from the tokens before it
    kv = B.paged_kv(c.k, c.v, c.table, c.lens, hq, None, c.status)
    meta, ref_meta = _meta(c, kind, lp), _meta(c, kind, lp)
    lens_now = c.lens.clone()
    old = _t([o for o, _ in spec])
    kv_old = B.paged_kv(c.k, c.v, c.table, old, hq, None, c.status)
    B.dsa_build_page_meta(kv_old, kind, lp, meta)
    B.dsa_build_page_meta(kv_old, kind, lp, ref_meta)
    before_k, before_v = c.k.clone(), c.v.clone()
    q_out = torch.full((T, hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    B.dsa_append_chunk(kv, chunk, k, v, rot_d, q, q_out, kind, lp, meta)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    # rotation: a value is rounded once to bf16 (2^-8 of itself), from fp32 products of values below 8
    # with sines off by at most 2^-21: 2^-17 in all
    for x, got in ((q, q_out), (k, None)):
        ref = rotate_reference(x[:live], positions[:, :live], axis, freq, inter)
        if got is None:
            got = torch.zeros(live, hkv, 128, dtype=torch.bfloat16, device="cuda")
            t = 0
            for b, (o, n) in enumerate(spec):
                for i in range(n):
                    got[t] = c.k[int(c.table[b, (o + i) // page]), :, (o + i) % page]
                    t += 1
        err = np.abs(got[:live].double().cpu().numpy() - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -16).all()
    assert (q_out[live:] == 3.0).all()
    # values are copied, nothing else in the pools changes
    t = 0
    for b, (o, n) in enumerate(spec):
        for i in range(n):
            ph, sl = int(c.table[b, (o + i) // page]), (o + i) % page
            assert torch.equal(c.v[ph, :, sl], v[t])
            before_k[ph, :, sl], before_v[ph, :, sl] = c.k[ph, :, sl], c.v[ph, :, sl]
            t += 1
    assert torch.equal(c.k.view(torch.int16), before_k.view(torch.int16))
    assert torch.equal(c.v.view(torch.int16), before_v.view(torch.int16))
    # metadata: the bits of a build over the whole cache, on touched pages only
    assert torch.equal(c.lens, lens_now)
    full = _meta(c, kind, lp)
    B.dsa_build_page_meta(kv, kind, lp, full)
    for b, (o, n) in enumerate(spec):
        for j in range(ceil_div(o + n, page)):
            if n and j >= o // page:
                ph = int(c.table[b, j])
                ref_meta[ph] = full[ph]
    bits = torch.int16 if kind == B.DSA_META_MINMAX else torch.int32
    assert torch.equal(meta.view(bits), ref_meta.view(bits))


def test_append_chunk_matches_the_single_token_append():
    """One token per request without rotation: the bits of dsa_append_kv, pools and metadata."""
    spec = [(63, 1), (64, 1), (7, 1)]
    out = []
    for chunked in (False, True):
        c = ChunkCase(spec, 64, 8, 2, seed=1)
        kv = B.paged_kv(c.k, c.v, c.table, c.lens, 8, None, c.status)
        meta = _meta(c, 0, 16)
        new = torch.randn(2, 3, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
        if chunked:
            B.dsa_append_chunk(kv, _chunk_of(c), new[0], new[1], meta_kind=0, logical_page=16,
                               meta=meta)
        else:
            B.dsa_append_kv(kv, new[0], new[1], 0, 16, meta)
        out.append([x.view(torch.int16).clone() for x in (c.k, c.v, meta)])
    for x, y in zip(*out):
        assert torch.equal(x, y)


def test_append_chunk_in_place_and_bad_pages():
    """q turned in place; tokens on a bad page write nothing, their queries are still turned."""
    c = ChunkCase([(0, 20), (10, 40)], 16, 4, 2, seed=4)
    kv = B.paged_kv(c.k, c.v, c.table, c.lens, 4, None, c.status)
    c.table[1, 2] = c.phys  # one past the pool
    c.table[0, 1] = -3
    k0 = c.k.clone()
    new = torch.randn(60, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    freq = [10000.0 ** (-i / 64) for i in range(64)]
    rot = B.rotary(B.rotary_phases(freq), 128)
    q, sep = c.q.clone(), torch.empty_like(c.q)
    chunk = _chunk_of(c)
    B.dsa_append_chunk(kv, chunk, new, new, rot, c.q, sep)
    B.dsa_append_chunk(kv, chunk, new, new, rot, q, q)
    torch.cuda.synchronize()
    assert torch.equal(q, sep) and int(c.status) == B.DSA_STATUS_BAD_PAGE
    pos = torch.cat([torch.arange(20), torch.arange(10, 50)])[None]
    ref = rotate_reference(c.q, pos, [0] * 64, freq, False)
    assert (np.abs(q.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -16).all()
    touched = {int(c.table[0, 0]), int(c.table[1, 0]), int(c.table[1, 1]), int(c.table[1, 3])}
    for ph in range(c.phys):
        if ph not in touched:
            assert torch.equal(c.k[ph].view(torch.int16), k0[ph].view(torch.int16))


@pytest.mark.parametrize("sign", [1, -1])
def test_append_turns_small_angles_to_the_last_bit(sign):
    """Angles of 2^-36 to 2^-22 of a turn on both sides of zero, where the sine alone decides the value:
    one half of every pair is zero, so the other half's place gets y sin.  The sine is off by 2^-24 of
    itself at most and the product by as much, so the stored value is the rounding of the exact one, or
    of what lies 2^-22 of it away."""
    n, p = 40, 16
    phase = [int(2 ** (28 + i * 14 / 64) / n) | 1 for i in range(64)]
    k, v = (torch.zeros(3, 1, p, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    new = torch.randn(n, 1, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    new[..., :64] = 0
    status = torch.zeros(1, dtype=I32, device="cuda")
    table, lens = _t([[0, 1, 2]]), _t([n])
    kv = B.paged_kv(k, v, table, lens, 1, None, status)
    rot = B.rotary(torch.tensor(phase, dtype=torch.int64, device="cuda"), 128,
                   positions=_t([[sign * (i + 1) for i in range(n)]]))
    chunk = B.chunk(_t([0, n]), _t([n]), _t([0] * n), _t(list(range(n))))
    B.dsa_append_chunk(kv, chunk, new, new, rot)
    torch.cuda.synchronize()
    assert int(status) == 0
    got = k.reshape(-1, 128)[:n].cpu()
    pos = np.array([sign * (i + 1) for i in range(n)], dtype=np.float64)[:, None]
    exact = -new[:, 0, 64:].double().cpu().numpy() * np.sin(
        pos * np.array(phase, dtype=np.float64) * (2 * np.pi / 2.0 ** 64))
    near = [torch.tensor(exact * (1 + e)).bfloat16() for e in (-2.0 ** -22, 2.0 ** -22)]
    assert ((got[:, :64] == near[0]) | (got[:, :64] == near[1])).all()
    # (the cosine is 1 there to far below 2^-24)
    assert torch.equal(got[:, 64:], new[:, 0, 64:].cpu())


# ----------------------------------------------------------------------------------------- attention

def _attend(c, scale=SCALE, sink=0, local=0, ws=None, stream=None):
    kv = B.paged_kv(c.k, c.v, c.table, c.lens, c.hq, c.streaming, c.status)
    T = c.tokens
    out = torch.full((T, c.hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    m, l = (torch.full((T, c.hq), 5.0, device="cuda") for _ in range(2))
    if ws is None:
        ws = torch.zeros(B.dsa_chunk_attn_workspace_size(kv, T), dtype=torch.uint8, device="cuda")
    B.dsa_chunk_attn(kv, B.chunk(c.start, c.count, tokens=T), c.q, scale, out, m, l, ws, sink, local,
                     stream)
    return out, m, l


DENSE = [
    # spec, page, hq, hkv
    ([(0, 1)], 16, 4, 1),
    ([(0, 1)], 256, 1, 1),
    ([(127, 1), (128, 1), (0, 2), (255, 1)], 16, 4, 1),
    ([(1000, 1), (17, 1), (0, 0), (300, 1)], 64, 8, 2),
    ([(5000, 1)], 16, 32, 2),
    ([(0, 128)], 16, 1, 1),
    ([(0, 129), (0, 127)], 32, 2, 2),
    ([(0, 64), (0, 65), (3, 63)], 48, 4, 1),
    ([(100, 33)], 16, 3, 1),
    ([(0, 300), (513, 77), (40, 1), (2, 0), (7, 5)], 16, 8, 2),
    ([(0, 257)], 112, 5, 1),
    ([(250, 40), (1, 90)], 80, 7, 1),
    ([(90, 150)], 240, 16, 1),
    ([(11, 31)], 128, 13, 1),
    ([(0, 700)], 16, 2, 2),
    ([(1500, 200)], 64, 6, 1),
    ([(i * 13, 1 + i % 3) for i in range(40)], 16, 4, 2),
    ([(i % 70, (i % 5) * (i % 3)) for i in range(600)], 16, 2, 1),
    ([(i % 90, (i % 4) * (i % 3)) for i in range(1100)], 16, 2, 2),
    ([(5000 - 100 * i, 1 + 70 * (i % 5 == 2)) for i in range(45)], 64, 4, 1),
    ([(200, 40)], 32, 80, 40),
    ([(70000, 16)], 64, 16, 1),    # 78 parts of a 256-row item
    ([(100000, 1), (3, 1)], 64, 8, 1),
]


@pytest.mark.parametrize("spec,page,hq,hkv", DENSE)
def test_chunk_attn_dense(spec, page, hq, hkv):
    c = ChunkCase(spec, page, hq, hkv, seed=11, extra_tokens=3)
    out, m, l = _attend(c)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    c.check(out, m, l, SCALE)
    live = sum(n for _, n in spec)
    assert (out[live:] == 5).all() and (m[live:] == 5).all() and (l[live:] == 5).all()


@pytest.mark.parametrize("sink,local", [(0, 0), (0, 1), (4, 0), (64, 256), (3, 100), (128, 128),
                                        (1, 1), (130, 17), (100000, 2), (2, 100000),
                                        ((1 << 31) - 1, (1 << 31) - 1)])
@pytest.mark.parametrize("spec,page,hq,hkv,streaming", [
    ([(0, 1), (500, 1), (1000, 3)], 16, 8, 2, [1, 1]),
    ([(0, 400), (700, 130)], 64, 4, 2, [0, 1]),
    ([(333, 260)], 48, 6, 3, [1, 0, 1]),
    ([(70, 3), (600, 1)], 16, 36, 36, [i % 3 == 1 for i in range(36)]),
])
def test_chunk_attn_streaming(spec, page, hq, hkv, streaming, sink, local):
    """Streaming heads beside dense ones, windows and sinks of every relation to the lengths; a window
    of no tokens leaves empty rows."""
    c = ChunkCase(spec, page, hq, hkv, seed=5, streaming=streaming)
    out, m, l = _attend(c, sink=sink, local=local)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    c.check(out, m, l, SCALE, (sink, local))


def test_chunk_attn_single_tokens_match_the_decode_calls():
    """One token per request: the rows of the sparse decode over all pages, and of the streaming
    decode (fp32 there, one bf16 rounding here)."""
    c = ChunkCase([(700, 1), (64, 1), (129, 1)], 16, 8, 2, seed=6, streaming=[0, 1])
    out, m, l = _attend(c, sink=16, local=100)
    kv = B.paged_kv(c.k, c.v, c.table, c.lens, 8, c.streaming, c.status)
    width = c.table.shape[1]
    idx = torch.arange(width, dtype=I32, device="cuda").expand(3, 2, width).contiguous()
    count = _t([[ceil_div(o + n, 16)] * 2 for o, n in c.spec])
    o2 = torch.zeros(3, 8, 128, device="cuda")
    m2, l2 = torch.zeros(3, 8, device="cuda"), torch.zeros(3, 8, device="cuda")
    ws = torch.zeros(max(16, B.dsa_sparse_decode_attn_workspace_size(kv, width)), dtype=torch.uint8,
                     device="cuda")
    B.dsa_sparse_decode_attn(kv, c.q, idx, count, SCALE, o2, m2, l2, workspace=ws)
    B.dsa_streaming_head_attn(kv, c.q, 16, 100, SCALE, o2, m2, l2)
    torch.cuda.synchronize()
    # both round every probability to bf16 (2^-8 of itself at most), once more the result here
    assert ((out.float() - o2).abs() <= 2.0 ** -8 * o2.abs() + 2.0 ** -7 * 4.5).all()
    assert (m - m2).abs().max() <= 1e-4 and ((l - l2).abs() <= 1e-3 * l2).all()


@pytest.mark.parametrize("seed", range(12))
def test_chunk_attn_random(seed):
    r = random.Random(seed)
    hkv, G = r.choice([(1, 1), (2, 4), (1, 8), (2, 3), (3, 2), (1, 16), (1, 11)])
    page = r.choice([16, 32, 48, 64, 128, 256])
    spec = [(r.choice([0, r.randint(0, 900)]), r.choice([0, 1, 1, r.randint(1, 20),
                                                        r.randint(1, 500)]))
            for _ in range(r.randint(1, 9))]
    if not any(n for _, n in spec):
        spec.append((3, 4))
    streaming = r.choice([None, [r.randint(0, 1) for _ in range(hkv)]])
    c = ChunkCase(spec, page, hkv * G, hkv, seed=seed, extra_tokens=r.choice([0, 7]),
                  streaming=streaming)
    sink, local = r.choice([0, 5, 64]), r.choice([1, 33, 300])
    scale = r.choice([SCALE, 1.0, 0.01])
    out, m, l = _attend(c, scale, sink, local)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    c.check(out, m, l, scale, (sink, local))


def test_chunk_attn_refused_requests_and_bad_pages():
    """Requests of count 0 leave their rows alone; the tokens of a bad page contribute nothing."""
    c = ChunkCase([(40, 60), (0, 30), (100, 1)], 16, 4, 2, seed=8)
    c.count[1] = 0  # refused: its 30 tokens stay on the axis
    c.lens[1] = 0
    bad = [(0, 2), (2, 0), (2, 6)]
    for b, j in bad:
        c.table[b, j] = c.phys + 5 if j else -1
    out, m, l = _attend(c)
    torch.cuda.synchronize()
    assert int(c.status) == B.DSA_STATUS_BAD_PAGE
    assert (out[60:90] == 5).all() and (m[60:90] == 5).all() and (l[60:90] == 5).all()
    from chunk_support import attend_reference, check_rows, visible
    for b in (0, 2):
        o, n = c.spec[b]
        L, t0 = o + n, int(c.start[b])
        ok = visible(np.arange(o, L), L, None)
        for bb, j in bad:
            if bb == b:
                ok[:, j * 16:(j + 1) * 16] = False
        c.table.clamp_(0, c.phys - 1)
        for hh in range(4):
            K, V = c.rows(c.k, b, hh // 2), c.rows(c.v, b, hh // 2)
            ref = attend_reference(c.q[t0:t0 + n, hh].double().cpu().numpy(), np.nan_to_num(K),
                                   np.nan_to_num(V), ok, SCALE)
            check_rows((out[t0:t0 + n, hh], m[t0:t0 + n, hh], l[t0:t0 + n, hh]), ref,
                       f"request {b} head {hh}")


def test_chunk_attn_tokens_outside_the_axis():
    """A chunk whose arrays point behind the token axis: a status, and nothing written outside."""
    c = ChunkCase([(40, 60), (10, 30)], 16, 4, 2, seed=8)
    kv = B.paged_kv(c.k, c.v, c.table, c.lens, 4, None, c.status)
    T = 70  # the axis ends inside request 1
    big = torch.full((c.tokens, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    m, l = (torch.full((c.tokens, 4), 5.0, device="cuda") for _ in range(2))
    ws = torch.zeros(B.dsa_chunk_attn_workspace_size(kv, T), dtype=torch.uint8, device="cuda")
    B.dsa_chunk_attn(kv, B.chunk(c.start, c.count, tokens=T), c.q[:T], SCALE, big[:T], m[:T], l[:T], ws)
    torch.cuda.synchronize()
    assert int(c.status) == B.DSA_STATUS_OVERFLOW
    assert (big[T:] == 5).all() and (m[T:] == 5).all()
    c.check(big, m, l, SCALE, requests=[0])


def test_chunk_attn_count_beyond_the_axis():
    """A request with more tokens than the axis: a status, and the rows that are there are right."""
    c = ChunkCase([(40, 90)], 16, 4, 2, seed=9)
    kv = B.paged_kv(c.k, c.v, c.table, c.lens, 4, None, c.status)
    T = 70
    big = torch.full((c.tokens, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    m, l = (torch.full((c.tokens, 4), 5.0, device="cuda") for _ in range(2))
    ws = torch.zeros(B.dsa_chunk_attn_workspace_size(kv, T), dtype=torch.uint8, device="cuda")
    B.dsa_chunk_attn(kv, B.chunk(c.start, c.count, tokens=T), c.q[:T], SCALE, big[:T], m[:T], l[:T], ws)
    torch.cuda.synchronize()
    assert int(c.status) == B.DSA_STATUS_OVERFLOW
    assert (big[T:] == 5).all() and (m[T:] == 5).all()
    c.spec[0] = (40, T)
    c.check(big, m, l, SCALE)


@pytest.mark.parametrize("batch", [16, 40])
def test_chunk_attn_counts_far_beyond_the_axis(batch):
    """Requests that each claim the whole axis, over tables of 2^30 positions: more key tiles than 32
    bits count.  A status, and nothing is written."""
    T, pages = 48000, 1 << 22
    table = torch.full((batch, pages), -1, dtype=torch.int32, device="cuda")
    pool = torch.zeros(4, 1, 256, 128, dtype=torch.bfloat16, device="cuda")
    lens = torch.full((batch,), 1 << 30, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = B.paged_kv(pool, pool, table, lens, 1, None, status)
    start = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    count = torch.full((batch,), T, dtype=torch.int32, device="cuda")
    q = torch.zeros(T, 1, 128, dtype=torch.bfloat16, device="cuda")
    out, m, l = torch.full_like(q, 5), *(torch.full((T, 1), 5.0, device="cuda") for _ in range(2))
    ws = torch.zeros(B.dsa_chunk_attn_workspace_size(kv, T), dtype=torch.uint8, device="cuda")
    B.dsa_chunk_attn(kv, B.chunk(start, count, tokens=T), q, SCALE, out, m, l, ws)
    torch.cuda.synchronize()
    assert int(status) == B.DSA_STATUS_OVERFLOW
    assert (out == 5).all() and (m == 5).all() and (l == 5).all() and not ws.any()


def test_chunk_attn_many_whole_items():
    """One prompt of many heads of their own: several whole items a CTA, of 2 to 22 key tiles."""
    n, heads = 2700, 64
    c = ChunkCase([(0, n)], 64, heads, heads, seed=10)
    out, m, l = _attend(c, SCALE)
    torch.cuda.synchronize()
    from chunk_support import attend_reference, check_rows, visible
    ok = visible(np.arange(n), n, None)
    for h in (0, 17, 63):
        ref = attend_reference(c.q[:, h].double().cpu().numpy(), c.rows(c.k, 0, h),
                               c.rows(c.v, 0, h), ok, SCALE)
        check_rows((out[:, h], m[:, h], l[:, h]), ref, f"head {h}")


def test_chunk_attn_large_logits():
    """Logits of several hundred, growing along the sequence (the running maximum moves at every tile)
    and falling (it never moves)."""
    for sign in (1, -1):
        c = ChunkCase([(600, 70)], 16, 4, 1, seed=2)
        L = 670
        u = torch.randn(128, generator=torch.Generator().manual_seed(1)).cuda()
        u = u / u.norm()
        c.q = (c.q.float() * 0.1 + 10 * u).bfloat16()
        for j in range(ceil_div(L, 16)):
            n = min(16, L - 16 * j)
            ramp = sign * (torch.arange(n, device="cuda") + 16 * j) * 0.1
            c.k[int(c.table[0, j]), 0, :n] += (ramp[:, None] * u).bfloat16()
        out, m, l = _attend(c, 1.0)
        torch.cuda.synchronize()
        c.check(out, m, l, 1.0)


def test_chunk_attn_nonfinite_rows_stay_apart():
    """A NaN query spoils its own row only; a NaN key spoils the rows that see it."""
    c = ChunkCase([(30, 100)], 16, 2, 1, seed=3)
    c.q[17, 1] = float("nan")
    pos = 30 + 60
    c.k[int(c.table[0, pos // 16]), 0, pos % 16, 5] = float("nan")
    out, m, l = _attend(c)
    torch.cuda.synchronize()
    bad = torch.zeros(100, 2, dtype=torch.bool, device="cuda")
    bad[17, 1] = True
    bad[60:] = True
    assert torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad)
    assert torch.equal(l.isnan(), bad)


def test_chunk_attn_reuses_a_workspace_and_runs_on_other_streams():
    """One workspace through calls of different shapes; the caller's stream is the one used."""
    cases = [ChunkCase([(3000, 1), (5, 200)], 16, 8, 2, seed=1), ChunkCase([(4000, 2)], 16, 8, 2, 2),
             ChunkCase([(0, 1)], 16, 8, 2, seed=3)]
    sizes = [B.dsa_chunk_attn_workspace_size(B.paged_kv(c.k, c.v, c.table, c.lens, 8), c.tokens)
             for c in cases]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [_attend(c, ws=ws) for c in cases for _ in range(2)]
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        c.check(*got[2 * i], SCALE)
        for x, y in zip(got[2 * i], got[2 * i + 1]):
            assert torch.equal(x, y)  # the same bits on every call


def test_step_in_a_graph_with_changing_lengths():
    """Plan, rotary append and attention of a step captured once and replayed with other lengths and
    tokens: each replay equals the eager calls on a copy of the state, and the reference."""
    from dynamic_block_sparse_gb300.pipeline import Cache, Chunk
    torch.manual_seed(0)
    hq, hkv, p, width, T = 8, 2, 16, 20, 96

    def state():
        k = torch.zeros(64, hkv, p, 128, dtype=torch.bfloat16, device="cuda")
        cache = Cache(k, k.clone(), torch.full((3, width), -1, dtype=I32, device="cuda"),
                      torch.zeros(3, dtype=I32, device="cuda"), hq)
        return cache, Chunk(cache, T, free_pages=torch.arange(64, dtype=I32, device="cuda"))

    freq = [10000.0 ** (-i / 64) for i in range(64)]
    rot = B.rotary(B.rotary_phases(freq), 128)
    qkv = torch.zeros(T, hq + 2 * hkv, 128, dtype=torch.bfloat16, device="cuda")
    delta = torch.zeros(3, dtype=I32, device="cuda")

    def step(cache, chunk):
        chunk.plan(delta)
        q = chunk.append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], rotary=rot, q=qkv[:, :hq])
        return chunk.attend(q)

    (ca, cha), (cb, chb) = state(), state()
    meta = ca.meta_buffer(B.DSA_META_MINMAX, 16)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(*state())  # attributes are set outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step(ca, cha)
    for d in ([40, 0, 50], [1, 1, 1], [30, 66, 0], [-20, 1, 1], [1, -100, 90]):
        delta.copy_(_t(d))
        qkv.copy_(torch.randn(qkv.shape, device="cuda").bfloat16())
        graph.replay()
        want = step(cb, chb)
        torch.cuda.synchronize()
        live = sum(max(x, 0) for x in d)
        for x, y in zip(got, want):
            assert torch.equal(x[:live], y[:live])
        for x, y in ((ca.page_table, cb.page_table), (ca.seq_lens, cb.seq_lens),
                     (ca.k_pages, cb.k_pages), (cha.free_count, chb.free_count)):
            assert torch.equal(x, y)
        assert int(ca.status) == 0 and int(cb.status) == 0
    assert meta.numel() > 0


def test_two_workspaces_on_two_streams_at_once():
    """Two calls that overlap on the GPU, each with its own workspace."""
    c = [ChunkCase([(5000, 3), (10, 100)], 16, 8, 2, seed=i) for i in (1, 2)]
    ref = [_attend(x) for x in c]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in c]
    got = []
    for _ in range(3):
        for x, s in zip(c, streams):
            with torch.cuda.stream(s):
                got.append(_attend(x))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for x, y in zip(g, ref[i % 2]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("spec", [
    [(12306, 1), (4948, 1), (0, 347), (0, 1), (4896, 1)],
    [(0, 389), (0, 312), (0, 320), (3231, 1)],
])
def test_chunk_attn_merges_wait_for_both_streams(spec):
    """32 heads of their own over requests whose cut leaves CTAs with a part of a long item and then a
    whole item of 129 to 256 tokens, in which the first 128 tokens see a key tile less than the others:
    the merge at the CTA's end may not begin before the later of the two is done.  The same bits on
    every call, alone and beside a call on another stream that delays some of the CTAs."""
    c = ChunkCase(spec, 64, 32, 32, seed=12)
    other = ChunkCase([(3000, 1), (0, 200)], 64, 8, 8, seed=13)
    ws = torch.zeros(B.dsa_chunk_attn_workspace_size(
        B.paged_kv(c.k, c.v, c.table, c.lens, 32), c.tokens), dtype=torch.uint8, device="cuda")
    first = _attend(c, ws=ws)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    c.check(*first, SCALE)
    s = torch.cuda.Stream()
    for rep in range(40):
        if rep % 2:
            with torch.cuda.stream(s):
                _attend(other)
        got = _attend(c, ws=ws)
        for x, y in zip(got, first):
            assert torch.equal(x, y)
    torch.cuda.synchronize()
    assert int(c.status) == 0 and int(other.status) == 0


# -------------------------------------------------------------------------------------- the pipeline

def test_step_in_a_pool_beyond_32_bit_offsets():
    """Pages whose elements lie behind 2^31 of the pool (4.3 GB each for keys and values)."""
    from chunk_support import attend_reference, check_rows, visible
    P = 65600
    k, v = (torch.zeros(P, 1, 256, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[65590, 3, 65599], [65598, 65597, 2]], dtype=torch.int32, device="cuda")
    spec = [(0, 600), (256, 44)]
    T = 644
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    row = [b for b, (o, n) in enumerate(spec) for _ in range(n)]
    pos = [o + i for o, n in spec for i in range(n)]
    chunk = B.chunk(i32([0, 600, T]), i32([600, 44]), i32(row), i32(pos))
    lens, status = i32([600, 300]), i32([0])
    g = torch.Generator().manual_seed(11)
    kn, vn, q = (torch.randn(T, h, 128, generator=g).bfloat16().cuda() for h in (1, 1, 2))
    kv = B.paged_kv(k, v, table, lens, 2, None, status)
    meta = torch.zeros(P, 1, 1, 128, 2, dtype=torch.bfloat16, device="cuda")
    B.dsa_append_chunk(kv, chunk, kn, vn, meta_kind=B.DSA_META_MINMAX, logical_page=256, meta=meta)
    out = torch.empty_like(q)
    m, l = (torch.empty(T, 2, device="cuda") for _ in range(2))
    ws = torch.zeros(B.dsa_chunk_attn_workspace_size(kv, T), dtype=torch.uint8, device="cuda")
    B.dsa_chunk_attn(kv, chunk, q, SCALE, out, m, l, ws)
    torch.cuda.synchronize()
    assert int(status) == 0
    for b, (o, n) in enumerate(spec):
        t0, L = (0, 600)[b], o + n
        K, V = (x[table[b].long(), 0].reshape(-1, 128)[:L] for x in (k, v))
        assert torch.equal(K[o:], kn[t0:t0 + n, 0]) and torch.equal(V[o:], vn[t0:t0 + n, 0])
        for j in range(o // 256, ceil_div(L, 256)):
            rows = K[256 * j:min(L, 256 * j + 256)]
            rec = meta[int(table[b, j]), 0, 0]
            assert torch.equal(rec[:, 0], rows.amax(0)) and torch.equal(rec[:, 1], rows.amin(0))
        ok = visible(np.arange(o, L), L, None)
        for h in range(2):
            ref = attend_reference(q[t0:t0 + n, h].double().cpu().numpy(), K.double().cpu().numpy(),
                                   V.double().cpu().numpy(), ok, SCALE)
            check_rows((out[t0:t0 + n, h], m[t0:t0 + n, h], l[t0:t0 + n, h]), ref,
                       f"request {b} head {h}")


def test_prefill_then_decode_through_the_decoders():
    """Prompts in two chunks through a decoder's prefill, then decode steps: metadata equals a fresh
    build bit for bit, and a decode step over all pages equals the attention of the chunk call."""
    from dynamic_block_sparse_gb300.pipeline import Cache, Chunk, HierDecoder, TopKDecoder
    torch.manual_seed(3)
    hq, hkv, p = 8, 2, 64
    for streaming in (None, [0, 1]):
        k = torch.zeros(80, hkv, p, 128, dtype=torch.bfloat16, device="cuda")
        hs = None if streaming is None else _t(streaming, torch.uint8)
        cache = Cache(k, k.clone(), torch.full((2, 12), -1, dtype=I32, device="cuda"),
                      torch.zeros(2, dtype=I32, device="cuda"), hq, hs)
        dec = (TopKDecoder(cache, k=12) if streaming is None else
               HierDecoder(cache, k_phys=12, logical_page=16, sink=32, local=100))
        chunk = Chunk(cache, 500, free_pages=torch.randperm(80, device="cuda").to(I32))
        rot = B.rotary(B.rotary_phases([10000.0 ** (-i / 64) for i in range(64)]), 128)
        for delta in ([300, 200], [77, 0], [1, 1], [1, 1]):
            n = sum(delta)
            qkv = torch.randn(500, hq + 2 * hkv, 128, device="cuda").bfloat16()
            chunk.plan(_t(delta))
            out, m, l = dec.prefill(chunk, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:],
                                    rotary=rot)
            torch.cuda.synchronize()
            assert int(cache.status) == 0
            fresh = torch.zeros_like(dec.meta)
            B.dsa_build_page_meta(cache.kv, B.DSA_META_MINMAX, dec.lp, fresh)
            for b in range(2):
                for j in range(ceil_div(int(cache.seq_lens[b]), p)):
                    ph = int(cache.page_table[b, j])
                    assert torch.equal(dec.meta[ph].view(torch.int16), fresh[ph].view(torch.int16))
            if delta == [1, 1]:
                q = chunk.q[:2].contiguous()
                o2, m2, l2 = dec.step(q) if streaming is None else dec.step(q, 0)
                # both round every probability and this one the result (2^-8 of itself each); values
                # of a few standard deviations bound the weighted sum of |v| by 4.5
                assert ((out[:2].float() - o2).abs() <= 2.0 ** -8 * o2.abs() + 2.0 ** -7 * 4.5).all()
                assert (m[:2] - m2).abs().max() <= 1e-4
            assert n >= 1


def test_hier_step_after_a_request_took_over_a_row():
    """A long request is released and a prompt takes its row between two selections: the step that would
    reuse the old selection attends the new request's pages, as a decoder without a past does."""
    from dynamic_block_sparse_gb300.pipeline import Cache, Chunk, HierDecoder
    torch.manual_seed(5)
    hq, hkv, p = 8, 2, 16
    k = torch.zeros(200, hkv, p, 128, dtype=torch.bfloat16, device="cuda")
    cache = Cache(k, k.clone(), torch.full((2, 80), -1, dtype=I32, device="cuda"),
                  torch.zeros(2, dtype=I32, device="cuda"), hq, _t([0, 1], torch.uint8))
    make = lambda: HierDecoder(cache, k_phys=4, logical_page=16, sink=8, local=40)
    dec = make()
    chunk = Chunk(cache, 1000, free_pages=torch.arange(200, dtype=I32, device="cuda"))
    new = lambda: [torch.randn(1000, h, 128, device="cuda").bfloat16() for h in (hq, hkv, hkv)]
    q = torch.randn(2, hq, 128, device="cuda").bfloat16()
    chunk.plan(_t([900, 60]))
    dec.prefill(chunk, *new())
    dec.step(q, 0)
    dec.idx[0].copy_(torch.tensor([40, 41, 42, 43], dtype=I32))  # the old request's far pages
    chunk.plan(_t([-900, 0]))
    chunk.plan(_t([200, 1]))
    dec.prefill(chunk, *new())
    got = [x.clone() for x in dec.step(q, 1)]
    fresh = make()
    fresh.build_meta()
    want = fresh.step(q, 0)
    torch.cuda.synchronize()
    assert int(cache.status) == 0
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert (got[2][0] > 0).all()


@pytest.mark.parametrize("fused", [True, False])
def test_prr_step_after_a_request_took_over_a_row(fused):
    """A request is released and a prompt takes its row between two PRR steps: the next step starts the
    predictor anew there and, in superset mode, attends the selected pages alone, while the other request
    (one more token, in a page that it had) carries its state on."""
    from dynamic_block_sparse_gb300.pipeline import Cache, Chunk, PRRDecoder, TopKDecoder
    torch.manual_seed(6)
    hq, hkv, p, k = 8, 2, 16, 4
    pool = torch.zeros(200, hkv, p, 128, dtype=torch.bfloat16, device="cuda")
    cache = Cache(pool, pool.clone(), torch.full((2, 80), -1, dtype=I32, device="cuda"),
                  torch.zeros(2, dtype=I32, device="cuda"), hq)
    dec = PRRDecoder(cache, k, 6, 0.3, 0.2, 0.5, superset=True, fused=fused)
    chunk = Chunk(cache, 1400, free_pages=torch.arange(200, dtype=I32, device="cuda"))
    new = lambda: [torch.randn(1400, h, 128, device="cuda").bfloat16() for h in (hq, hkv, hkv)]
    query = lambda: torch.randn(2, hq, 128, device="cuda").bfloat16()
    chunk.plan(_t([900, 500]))
    dec.prefill(chunk, *new())
    assert chunk.count.tolist() == [900, 500]
    for _ in range(3):
        dec.step(query())
    chunk.plan(_t([-900, 0]))
    chunk.plan(_t([300, 1]))
    ell = dec.ell.clone()
    dec.prefill(chunk, *new())
    assert torch.equal(dec.ell[1, :, :32], ell[1, :, :32])
    assert dec.spec_count.tolist() == [[0] * hkv, [6] * hkv]
    q = query()
    dec.step(q)
    one = TopKDecoder(cache, k)
    one.build_meta()
    want = one.step(q)
    torch.cuda.synchronize()
    assert int(cache.status) == 0
    assert torch.equal(dec.ell[0, :, :19], dec.scores[0, :, :19]) and (dec.trend[0] == 0).all()
    assert (dec.ell[0, :, 19:] == -math.inf).all()
    assert not torch.equal(dec.ell[1, :, :32], dec.scores[1, :, :32])
    assert torch.equal(dec.idx[0], one.idx[0])
    # the same pages, merged in another order: fp32 sums of some tens of tokens, and probabilities
    # rounded to bf16 against another maximum (2^-8 of themselves in both; |v| averages below 4.5)
    for x, y in zip((dec.out, dec.m, dec.l), want):
        assert (x[0] - y[0]).abs().max() <= 2.0 ** -7 * 4.5
    assert ((dec.l[0] - want[2][0]).abs() <= 2.0 ** -18 * want[2][0] * 64).all()


@pytest.mark.parametrize("name", ["topk", "threshold", "prr"])
def test_prefill_without_windows_attends_every_head(name):
    """Decoders that know no window prefill streaming heads over the whole cache as well: the rows of a
    cache without the marks, bit for bit."""
    from dynamic_block_sparse_gb300.pipeline import (Cache, Chunk, PRRDecoder, ThresholdDecoder,
                                                     TopKDecoder)
    make = {"topk": lambda c: TopKDecoder(c, 4), "threshold": lambda c: ThresholdDecoder(c, 0.9, 8),
            "prr": lambda c: PRRDecoder(c, 4, 6, 0.3, 0.2, 0.5)}[name]
    hq, hkv, p, T = 8, 2, 32, 300
    g = torch.Generator().manual_seed(7)
    new = [torch.randn(T, h, 128, generator=g).bfloat16().cuda() for h in (hq, hkv, hkv)]
    got = []
    for marks in (None, [0, 1], [0, 0], [1, 1]):
        k = torch.zeros(20, hkv, p, 128, dtype=torch.bfloat16, device="cuda")
        cache = Cache(k, k.clone(), torch.full((2, 9), -1, dtype=I32, device="cuda"),
                      torch.zeros(2, dtype=I32, device="cuda"), hq,
                      None if marks is None else _t(marks, torch.uint8))
        chunk = Chunk(cache, T, free_pages=torch.arange(20, dtype=I32, device="cuda"))
        chunk.plan(_t([200, 100]))
        got.append(make(cache).prefill(chunk, *new))
        torch.cuda.synchronize()
        assert int(cache.status) == 0
    assert (got[0][2] >= 1 - 2.0 ** -18).all()  # (the largest logit adds 1)
    for x in got[1:]:
        for a, b in zip(x, got[0]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["threshold", "prr"])
def test_prefill_then_decode_through_the_other_decoders(name):
    """Prompts in two chunks, a rollback and single tokens through the prefill of the PSA and PRR
    decoders, each followed by a decode step whose budget covers every page: metadata equals a fresh
    build bit for bit, and the step the rows that the chunk call gave the last tokens."""
    from dynamic_block_sparse_gb300.pipeline import Cache, Chunk, PRRDecoder, ThresholdDecoder
    torch.manual_seed(4)
    hq, hkv, p = 8, 2, 64
    k = torch.zeros(40, hkv, p, 128, dtype=torch.bfloat16, device="cuda")
    cache = Cache(k, k.clone(), torch.full((2, 12), -1, dtype=I32, device="cuda"),
                  torch.zeros(2, dtype=I32, device="cuda"), hq)
    if name == "threshold":
        dec, kind = ThresholdDecoder(cache, tau=1.0, cap=12), B.DSA_META_MEAN
    else:
        dec, kind = PRRDecoder(cache, 12, 12, 0.3, 0.2, 0.5), B.DSA_META_MINMAX
    chunk = Chunk(cache, 500, free_pages=torch.randperm(40, device="cuda").to(I32))
    rot = B.rotary(B.rotary_phases([10000.0 ** (-i / 64) for i in range(64)]), 128)
    lens = [0, 0]
    for delta in ([300, 200], [77, 1], [-100, -200], [1, 60], [1, 1]):
        chunk.plan(_t(delta))
        lens = [max(0, a + d) for a, d in zip(lens, delta)]
        if min(delta) < 0:
            continue
        qkv = torch.randn(500, hq + 2 * hkv, 128, device="cuda").bfloat16()
        out, m, l = dec.prefill(chunk, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], rotary=rot)
        torch.cuda.synchronize()
        assert int(cache.status) == 0 and cache.seq_lens.tolist() == lens
        fresh = torch.zeros_like(dec.meta)
        B.dsa_build_page_meta(cache.kv, kind, p, fresh)
        for b in range(2):
            for j in range(ceil_div(lens[b], p)):
                ph = int(cache.page_table[b, j])
                assert torch.equal(dec.meta[ph].view(torch.uint8), fresh[ph].view(torch.uint8))
        last = [delta[0] - 1, sum(delta) - 1]
        o2, m2, l2 = dec.step(chunk.q[last].contiguous())
        torch.cuda.synchronize()
        assert int(cache.status) == 0
        # both round every probability and this one the result (2^-8 of itself each); values of a few
        # standard deviations bound the weighted sum of |v| by 4.5
        assert ((out[last].float() - o2).abs() <= 2.0 ** -8 * o2.abs() + 2.0 ** -7 * 4.5).all()
        assert (m[last] - m2).abs().max() <= 1e-4


def test_captured_append_keeps_metadata():
    """Plan and append with both kinds of metadata captured once and replayed for other lengths: the
    records of every page that holds a token equal a fresh build's bit for bit."""
    from dynamic_block_sparse_gb300.pipeline import Cache, Chunk
    torch.manual_seed(1)
    hkv, p, T = 2, 32, 120
    k = torch.zeros(40, hkv, p, 128, dtype=torch.bfloat16, device="cuda")
    cache = Cache(k, k.clone(), torch.full((3, 10), -1, dtype=I32, device="cuda"),
                  torch.zeros(3, dtype=I32, device="cuda"), 4)
    chunk = Chunk(cache, T, free_pages=torch.arange(40, dtype=I32, device="cuda"))
    metas = [(kind, lp, cache.meta_buffer(kind, lp)) for kind, lp in (
        (B.DSA_META_MINMAX, 16), (B.DSA_META_MEAN, 32))]
    kn, vn = (torch.zeros(T, hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    delta = torch.zeros(3, dtype=I32, device="cuda")
    s = torch.cuda.Stream()

    def step():
        chunk.plan(delta)
        chunk.append(kn, vn, metas)

    with torch.cuda.stream(s):
        step()  # attributes are set outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for d in ([40, 0, 50], [1, 1, 1], [30, 66, 0], [-20, 1, 1], [1, -100, 90], [5, 33, 2]):
        delta.copy_(_t(d))
        for x in (kn, vn):
            x.copy_(torch.randn(x.shape, device="cuda").bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert int(cache.status) == 0
        for kind, lp, meta in metas:
            fresh = torch.zeros_like(meta)
            B.dsa_build_page_meta(cache.kv, kind, lp, fresh)
            for b in range(3):
                # (a page that a rollback shortened keeps its records until it gets a token)
                if d[b] > 0:
                    for j in range(ceil_div(int(cache.seq_lens[b]), p)):
                        ph = int(cache.page_table[b, j])
                        assert torch.equal(meta[ph].view(torch.uint8), fresh[ph].view(torch.uint8))


def test_rotary_with_a_strided_axis_list():
    """Axes given as a view turn as their dense copy does."""
    c = ChunkCase([(0, 40)], 16, 2, 1, seed=14)
    axis = (torch.arange(128, device="cuda") % 3).to(torch.uint8)[::2]
    pos = torch.randint(0, 1000, (3, 40), device="cuda").to(I32)
    phase = B.rotary_phases([10000.0 ** (-i / 64) for i in range(64)])
    got = []
    for a in (axis, axis.contiguous()):
        kv = B.paged_kv(c.k, c.v, c.table, c.lens, 2, None, c.status)
        chunk = B.chunk(c.start, c.count, _t([0] * 40), _t(list(range(40))))
        out = torch.empty_like(c.q)
        B.dsa_append_chunk(kv, chunk, c.q[:, :1], c.q[:, 1:], B.rotary(phase, 128, a, pos), c.q, out)
        got.append(out)
    torch.cuda.synchronize()
    assert int(c.status) == 0 and torch.equal(*got)
