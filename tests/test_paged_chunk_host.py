"""CPU-only checks of the chunk operators' host side: struct layouts, argument checks that answer
before any CUDA call, the fixed-point phases, and the reference page plan the GPU tests compare with
(its own invariants: pages are neither lost nor handed out twice)."""

import ctypes
import math
import os
import random
import subprocess

import numpy as np
import pytest
import torch

from chunk_support import plan_reference

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from dynamic_block_sparse_gb300 import binding, build
    build.build()
    return binding.load()


def _kv(**kw):
    from dynamic_block_sparse_gb300 import binding as B
    kv = B.PagedKV()
    kv.k_pages = kv.v_pages = kv.page_table = kv.seq_lens = 4096
    kv.batch, kv.num_q_heads, kv.num_kv_heads = 2, 8, 2
    kv.head_dim, kv.page_size, kv.max_pages_per_seq, kv.num_phys_pages = 128, 64, 8, 16
    for k, v in kw.items():
        setattr(kv, k, v)
    return kv


def _chunk(tokens=16, **kw):
    from dynamic_block_sparse_gb300 import binding as B
    c = B.Chunk()
    c.start = c.count = c.row = c.pos = c.slot = 4096
    c.tokens = tokens
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_struct_layouts_match_the_header(tmp_path):
    from dynamic_block_sparse_gb300 import binding as B
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "dsa.h"', "int main(void) {"]
    for cname, cls in (("dsa_chunk", B.Chunk), ("dsa_rotary", B.Rotary)):
        lines.append(f'  printf("{cname} %zu\\n", sizeof({cname}));')
        for f, _ in cls._fields_:
            lines.append(f'  printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));')
    lines += [f'  printf("no_pages %d\\n", DSA_STATUS_NO_PAGES);', "  return 0;", "}"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines) + "\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)],
                   check=True)
    got = dict(ln.split() for ln in subprocess.run([str(exe)], capture_output=True, text=True,
                                                    check=True).stdout.splitlines())
    assert int(got["no_pages"]) == B.DSA_STATUS_NO_PAGES
    for cname, cls in (("dsa_chunk", B.Chunk), ("dsa_rotary", B.Rotary)):
        assert int(got[cname]) == ctypes.sizeof(cls), cname
        for f, _ in cls._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(cls, f).offset, f"{cname}.{f}"


def test_plan_chunk_refusals(lib):
    def call(kv=None, chunk=None, lens=4096, delta=4096, free=4096, cap=16, fin=4096, fout=4096,
             ws=8192, ws_bytes=16):
        return lib.dsa_plan_chunk(ctypes.byref(kv or _kv()), lens, delta, free, cap, fin, fout,
                                  None if chunk == 0 else ctypes.byref(chunk or _chunk()), ws,
                                  ws_bytes, None)
    assert call(chunk=0) == -1
    assert call(chunk=_chunk(tokens=-1)) == -1
    assert call(cap=-1) == -1
    for name in ("lens", "delta", "free", "fin", "fout"):
        assert call(**{name: None}) == -1, name
    assert call(chunk=_chunk(start=None)) == -1
    assert call(chunk=_chunk(count=None)) == -1
    assert call(chunk=_chunk(row=None)) == -1
    assert call(chunk=_chunk(pos=None)) == -1
    assert call(kv=_kv(batch=8193)) == -3 and b"8193" in lib.dsa_last_error()
    assert call(kv=_kv(batch=8192, max_pages_per_seq=1 << 19)) == -3
    assert call(kv=_kv(page_size=256, max_pages_per_seq=1 << 23, batch=1)) == -3
    assert call(kv=_kv(page_size=256, max_pages_per_seq=(1 << 23) - 1, batch=1)) == -3
    assert call(ws=None) == -5
    assert call(ws_bytes=8) == -5
    assert call(ws=8200) == -2
    assert lib.dsa_plan_chunk_workspace_size(8) == 16


def test_append_chunk_refusals(lib):
    from dynamic_block_sparse_gb300 import binding as B

    def rot(**kw):
        r = B.Rotary()
        r.phase, r.num_axes, r.rot_dim = 4096, 1, 128
        for k, v in kw.items():
            setattr(r, k, v)
        return r

    def call(kv=None, chunk=None, k=8192, ks=256, v=8192, vs=256, rotary=None, q=None, qs=1024,
             qo=None, kind=0, lp=16, meta=16384):
        return lib.dsa_append_chunk(
            ctypes.byref(kv or _kv()), None if chunk == 0 else ctypes.byref(chunk or _chunk()), k,
            ks, v, vs, None if rotary is None else ctypes.byref(rotary), q, qs, qo, kind, lp, meta,
            None)
    assert call(chunk=0) == -1
    assert call(chunk=_chunk(tokens=-1)) == -1
    assert call(chunk=_chunk(tokens=0), k=None) == 0                 # nothing to do
    assert call(k=None) == -1 and call(v=None) == -1
    for f in ("start", "count", "row", "pos"):
        assert call(chunk=_chunk(**{f: None})) == -1, f
    assert call(k=8200) == -2 and call(v=8200) == -2
    assert call(ks=255) == -1 and call(ks=260) == -1 and call(vs=128) == -1
    assert call(q=4096) == -1 and call(qo=4096) == -1                # only together
    assert call(q=4100, qo=8192) == -2
    assert call(q=4096, qo=8192, qs=1023) == -1 and call(q=4096, qo=8192, qs=1028) == -1
    assert call(q=4096, qo=4096, qs=2048) == -1                      # in place needs contiguity
    assert call(rotary=rot(phase=None)) == -1
    assert call(rotary=rot(phase=4100)) == -2
    for bad in (0, 8, 24, 136, 144):
        assert call(rotary=rot(rot_dim=bad)) == -3, bad
    assert call(rotary=rot(num_axes=0)) == -3 and call(rotary=rot(num_axes=5)) == -3
    assert call(rotary=rot(num_axes=2)) == -1                        # axis and positions missing
    assert call(rotary=rot(num_axes=2, axis=4096)) == -1
    assert call(kind=2) == -1 and call(lp=48) == -1 and call(meta=16392) == -2


def test_chunk_attn_refusals(lib):
    def call(kv=None, chunk=None, q=4096, sink=0, local=0, scale=0.1, out=8192, ws=16384,
             ws_bytes=1 << 40):
        return lib.dsa_chunk_attn(ctypes.byref(kv or _kv()),
                                  None if chunk == 0 else ctypes.byref(chunk or _chunk()), q, sink,
                                  local, scale, out, None, None, ws, ws_bytes, None)
    assert call(chunk=0) == -1
    assert call(chunk=_chunk(tokens=-3)) == -1
    assert call(chunk=_chunk(tokens=0), q=None) == 0                 # nothing to do
    assert call(q=None) == -1 and call(out=None) == -1
    assert call(chunk=_chunk(start=None)) == -1 and call(chunk=_chunk(count=None)) == -1
    assert call(q=4104) == -2 and call(out=8200) == -2
    assert call(q=8192) == -1                                        # out may not be q
    assert call(sink=-1) == -1 and call(local=-1) == -1
    for bad in (0.0, -0.1, math.inf, -math.inf, math.nan, 1e-45, 3e38):
        assert call(scale=bad) == -1, bad
    assert call(ws=None) == -5 and call(ws_bytes=0) == -5 and call(ws=16392) == -2
    assert call(kv=_kv(head_dim=64)) == -3
    assert call(kv=_kv(page_size=256, max_pages_per_seq=1 << 23, batch=1)) == -3
    assert call(kv=_kv(batch=8193)) == -3
    # more than 2^31 key tiles, were every query at the end of its table
    assert call(kv=_kv(page_size=256, max_pages_per_seq=1 << 22, batch=1), chunk=_chunk(1 << 20)) == -3


def test_binding_refuses_wrong_tensors(lib):
    from dynamic_block_sparse_gb300 import binding as B
    z = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError, match="int32"):
        B.chunk(torch.zeros(3, dtype=torch.int64), z(2), z(4), z(4))
    with pytest.raises(ValueError, match="shape"):
        B.chunk(z(4), z(2), z(4), z(4))
    with pytest.raises(ValueError, match="CUDA"):
        B.chunk(z(3), z(2), z(4), z(4))
    with pytest.raises(ValueError, match="phase"):
        B.rotary(torch.zeros(32, dtype=torch.int64), 128)
    with pytest.raises(ValueError, match="contiguous"):
        B._token_rows(torch.zeros(4, 2, 256, dtype=torch.bfloat16)[..., ::2], 4, 2, "k_new")
    with pytest.raises(ValueError, match="bf16"):
        B._token_rows(torch.zeros(4, 2, 128), 4, 2, "k_new")
    assert B._token_rows(torch.zeros(4, 10, 128, dtype=torch.bfloat16)[:, 2:4], 4, 2, "k") == 1280
    kv, c = B.PagedKV(), B.Chunk()
    kv.batch, kv.num_phys_pages, kv.num_kv_heads, kv.page_size = 2, 3, 2, 32
    c.batch, c.tokens = 2, 4
    new = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    for short in (torch.zeros(3 * 2 * 2 * 256 - 1, dtype=torch.bfloat16),
                  torch.zeros(3 * 2 * 2 * 256, 2, dtype=torch.bfloat16)[:, 0]):
        with pytest.raises(ValueError, match="meta"):
            B.dsa_append_chunk(kv, c, new, new, logical_page=16, meta=short)
    with pytest.raises(ValueError, match="CUDA"):
        B.dsa_append_chunk(kv, c, new, new, logical_page=16,
                           meta=torch.zeros(3 * 2 * 2 * 256, dtype=torch.bfloat16))


def test_rotary_phases_are_exact_fractions_of_a_turn():
    """phase * position modulo 2^64 is the turn of position * frequency: checked against a 40-digit
    value of the angle at positions where float32 has lost it."""
    from fractions import Fraction

    from dynamic_block_sparse_gb300 import binding as B
    freqs = [500000.0 ** (-2 * i / 128) for i in range(64)] + [math.pi, 7.0]
    ph = B.rotary_phases(freqs, "cpu")
    two_pi = Fraction(62831853071795864769252867665590057683943, 10 ** 40)
    for f, p in zip(freqs, ph.tolist()):
        for pos in (0, 1, 131071, (1 << 31) - 1, -5):
            turns = Fraction(f) * pos / two_pi
            got = Fraction((p * pos) % 2 ** 64, 2 ** 64)
            off = abs(got - turns % 1)
            off = min(off, 1 - off)
            assert off <= Fraction(abs(pos) + 1, 2 ** 64), (f, pos)


@pytest.mark.parametrize("seed", range(20))
def test_plan_reference_keeps_every_page_once(seed):
    """Steps of random growth, rollback and release through the reference plan: at any time the pages
    of the live requests and the stack are a permutation of the pool."""
    r = random.Random(seed)
    p, B, width, phys = r.choice([16, 48]), r.randint(1, 9), r.randint(2, 12), r.randint(6, 60)
    table = np.full((B, width), -7, dtype=np.int64)
    lens, free = [0] * B, list(r.sample(range(phys), phys))
    seen = set()
    for _ in range(30):
        delta = [r.choice([0, 1, 1, r.randint(1, p * 3), -r.randint(1, 40), -10 ** 6])
                 for _ in range(B)]
        got = plan_reference(table, lens, delta, free, p, tokens=200)
        table, lens, free = got["table"], got["lens"], got["stack"]
        held = [int(table[b, j]) for b in range(B) for j in range(-(-lens[b] // p))]
        assert sorted(held + free) == list(range(phys))
        for t, (b, pos, slot) in enumerate(zip(got["row"], got["pos"], got["slot"])):
            if b >= 0:
                assert slot == table[b, pos // p] * p + pos % p and pos < lens[b]
                assert got["start"][b] <= t < got["start"][b] + got["count"][b]
            else:
                assert pos == slot == -1
        seen.add(got["refused"])
    assert seen  # both outcomes occur over the seeds; each is asserted page by page above


def test_prefill_is_refused_on_quantised_pages():
    """KV8 and KV4 pages are a copy of the pools: a prompt that entered the pools only would be missing
    from every later step."""
    from dynamic_block_sparse_gb300.pipeline import TopKDecoder
    for which in ("kv8", "kv4"):
        dec = object.__new__(TopKDecoder)
        dec.kv8 = dec.kv4 = None
        setattr(dec, which, torch.zeros(1, dtype=torch.uint8))
        with pytest.raises(ValueError, match="quantised"):
            dec.prefill(None, None, None, None)


def test_a_reused_selection_ends_with_a_prefill():
    """HierDecoder keeps its selection for ``reuse`` steps, but not across a prefill."""
    from dynamic_block_sparse_gb300.pipeline import HierDecoder

    class Chunk:
        def append(self, *a):
            return None

        def attend(self, *a, **kw):
            return None

    dec = object.__new__(HierDecoder)
    dec.reuse, dec.prefilled, dec.lp, dec.sink, dec.local, dec.scale = 4, False, 16, 1, 1, 1.0
    dec.cache = dec.meta = dec.out = dec.m = dec.l = None
    selected = []
    dec.attend = lambda q, stream=None: None

    def select(q, stream=None):
        selected.append(q)
        dec.prefilled = False

    dec.select = select
    for t in range(8):
        if t in (2, 4, 7):
            dec.prefill(Chunk(), None, None, None)
        dec.step(t, t)
    assert selected == [0, 2, 4, 7]


def test_the_predictor_forgets_pages_a_prefill_filled():
    """PRRDecoder: requests that grow, grow after a rollback, take over a row, or take no part."""
    import types

    from dynamic_block_sparse_gb300.pipeline import PRRDecoder
    dec = object.__new__(PRRDecoder)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)
    dec.cache = types.SimpleNamespace(seq_lens=i32([70, 48, 30, 0, 90]), page_size=16, device="cpu")
    dec.k_pred, dec.stride, dec.t = 4, 7, 3
    dec.ell = torch.arange(5 * 2 * 7).reshape(5, 2, 7).float()
    dec.trend = dec.ell + 1
    P = i32([[0, 2, 4, 5], [1, 3, 6, -1], [0, 1, 2, 3], [0, 3, -1, -1], [2, 3, 5, 6]])
    dec.spec_bufs = [None, P[:, None].expand(5, 2, 4).contiguous()]
    dec.spec_counts = [None, i32([[4] * 2, [3] * 2, [4] * 2, [2] * 2, [4] * 2])]
    ell, trend = dec.ell.clone(), dec.trend.clone()
    # tokens before the chunk: 65 (5 pages), 32 (2), 0, a refused request's 0, a request at rest
    dec._forget(types.SimpleNamespace(count=i32([5, 16, 30, 0, 0])))
    for b, kept in enumerate([5, 2, 0, 7, 7]):
        assert torch.equal(dec.ell[b, :, :kept], ell[b, :, :kept])
        assert torch.equal(dec.trend[b, :, :kept], trend[b, :, :kept])
        assert (dec.ell[b, :, kept:] == -math.inf).all() and (dec.trend[b, :, kept:] == 0).all()
    assert dec.spec_count.tolist() == [[3] * 2, [1] * 2, [0] * 2, [2] * 2, [4] * 2]


@pytest.mark.parametrize("name", ["TopKDecoder", "ThresholdDecoder", "PRRDecoder"])
def test_prefill_without_a_window_covers_the_cache(name):
    """These decoders have no sink and window to give: their prefill lets streaming heads see the whole
    cache, as its documentation says, instead of nothing."""
    import types

    from dynamic_block_sparse_gb300 import pipeline
    seen = {}

    class Chunk(pipeline.Chunk):
        def __init__(self, cache):
            self.cache = cache

        def append(self, *a):
            return "q"

        def attend(self, q, scale, sink=0, local=0, stream=None):
            seen.update(q=q, sink=sink, local=local)
            return "answer"

    cls = getattr(pipeline, name)
    dec = object.__new__(cls)
    dec.cache = types.SimpleNamespace(page_size=16, max_pages=9)
    dec.kind = dec.lp = dec.meta = None
    dec.scale = 1.0
    dec._forget = lambda *a: None
    assert dec.prefill(Chunk(dec.cache), None, None, None) == "answer"
    assert seen == dict(q="q", sink=144, local=0)


def test_overlapping_arguments_are_refused(lib):
    """An output that shares memory with an input or another output: the CTAs of a launch would read
    what others have written."""
    from dynamic_block_sparse_gb300 import binding as B
    at = lambda i: (1 << 32) + (i << 24)  # 16 MB apart
    kv = _kv(k_pages=at(30), v_pages=at(31), page_table=at(0), seq_lens=at(1))

    def refused(rc):
        return rc == -1 and b"overlap" in lib.dsa_last_error()

    def plan(**kw):
        a = dict(lens=at(2), delta=at(3), free=at(4), fin=at(5), fout=at(6), start=at(7), count=at(8),
                 row=at(9), pos=at(10), slot=at(11), ws=at(12))
        a.update(kw)
        c = _chunk(16, **{k: a[k] for k in ("start", "count", "row", "pos", "slot")})
        return lib.dsa_plan_chunk(ctypes.byref(kv), a["lens"], a["delta"], a["free"], 16, a["fin"],
                                  a["fout"], ctypes.byref(c), a["ws"], 16, None)
    for bad in (dict(delta=at(8)), dict(delta=at(8) + 4), dict(delta=at(1)), dict(lens=at(8)),
                dict(lens=at(1) + 4), dict(lens=at(9) + 60), dict(fin=at(4)), dict(pos=at(9)),
                dict(slot=at(9) + 32), dict(row=at(7) + 8), dict(free=at(0)), dict(fout=at(1)),
                dict(delta=at(12)), dict(count=at(7) - 4)):
        assert refused(plan(**bad)), bad

    def append(tokens=16, k=at(2), v=at(3), q=at(4), qs=1024, qo=at(5), ks=256):
        return lib.dsa_append_chunk(ctypes.byref(kv), ctypes.byref(_chunk(tokens)), k, ks, v, 256, None,
                                    q, qs, qo, 0, 16, None, None)
    assert refused(append(qo=at(4) + 16)) and refused(append(qo=at(2))) and refused(append(qo=at(3)))
    assert refused(append(qo=at(4) + 16 * 2048 - 16)) and refused(append(qo=at(2) - 16 * 2048 + 16))
    # slices of one projection of 13 heads, q_out over the last token's k
    assert refused(append(q=at(4), qs=1664, k=at(4) + 2048, ks=1664, qo=at(4) + 15 * 3328 + 2544))

    def attend(q=at(2), out=at(3), m=at(4), l=at(5), ws=at(6)):
        return lib.dsa_chunk_attn(ctypes.byref(kv), ctypes.byref(_chunk(16)), q, 0, 0, 0.1, out, m, l,
                                  ws, 1 << 30, None)
    for bad in (dict(out=at(2) + 16), dict(out=at(2) - 16), dict(m=at(2)), dict(l=at(3) + 32764),
                dict(m=at(5)), dict(ws=at(2) - 4096), dict(l=at(6)), dict(l=at(4) + 508)):
        assert refused(attend(**bad)), bad


def test_current_stream_without_the_short_cuts():
    """The stream's handle comes from torch's public calls where torch has no shorter ones."""
    import sys
    code = """
import types, torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda device=None: types.SimpleNamespace(cuda_stream=100 + (device or 0))
from dynamic_block_sparse_gb300 import binding as B
assert B._stream(None) in (100, 103) and B._stream(types.SimpleNamespace(cuda_stream=7)) == 7
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


class _OnDevice:
    """A tensor's look on a CUDA device that is not there."""

    def __init__(self, t, device: int):
        self.t, self.dtype, self.shape, self.nbytes = t, t.dtype, t.shape, t.nbytes
        self.device, self.is_cuda = torch.device("cuda", device), True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 1 << 32

    def is_contiguous(self):
        return True

    def contiguous(self):
        return self

    def numel(self):
        return self.t.numel()


def test_tensors_of_another_device_are_refused(lib, monkeypatch):
    """Every tensor of the three calls, those of the descriptors among them, has to be on the current
    device: a kernel there could not read it."""
    import types

    from dynamic_block_sparse_gb300 import binding as B
    monkeypatch.setattr(B, "_device", lambda: 0)
    calls = []
    ran = types.SimpleNamespace(**{n: lambda *a, n=n: calls.append(n) or 0 for n in (
        "dsa_plan_chunk", "dsa_append_chunk", "dsa_chunk_attn")})
    monkeypatch.setattr(B, "load", lambda: ran)
    T, bf = 6, torch.bfloat16
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    rows = lambda h: torch.zeros(T, h, 128, dtype=bf)
    stream = types.SimpleNamespace(cuda_stream=1)

    def run(call, other=()):
        d = lambda name, t: _OnDevice(t, 1 if name in other else 0)
        pool = lambda n: d("kv", torch.zeros(4, 2, 16, 128, dtype=bf))
        chunk = B.chunk(*(d("chunk", x) for x in (i32(3), i32(2), i32(T), i32(T))))
        kv = B.paged_kv(pool(0), pool(1), d("kv", i32(2, 3)), d("kv", i32(2)), 4)
        if call == "plan":
            kv = B.page_tables(d("kv", i32(2, 3)), d("kv", i32(2)), 16, 4)
            B.dsa_plan_chunk(kv, d("lens_in", i32(2)), d("delta", i32(2)), d("free_pages", i32(4)),
                             d("free_in", i32(1)), d("free_out", i32(1)), chunk,
                             d("workspace", i32(4)), stream)
        elif call == "append":
            rot = B.rotary(d("rotary", torch.zeros(64, dtype=torch.int64)), 128)
            B.dsa_append_chunk(kv, chunk, d("k_new", rows(2)), d("v_new", rows(2)), rot,
                               d("q", rows(4)), d("q_out", rows(4)), 0, 16,
                               d("meta", torch.zeros(4 * 2 * 256, dtype=bf)), stream)
        else:
            f32 = torch.zeros(T, 4)
            B.dsa_chunk_attn(kv, chunk, d("q", rows(4)), 0.1, d("out", rows(4)), d("m", f32),
                             d("l", f32), d("workspace", i32(4)), 0, 0, stream)

    names = {"plan": "kv chunk lens_in delta free_pages free_in free_out workspace",
             "append": "kv chunk k_new v_new rotary q q_out meta", "attend": "kv chunk q out m l workspace"}
    for call, args in names.items():
        run(call)
        assert len(calls) == 1
        for name in args.split():
            with pytest.raises(ValueError, match="current CUDA device"):
                run(call, (name,))
        assert len(calls) == 1, call
        calls.clear()
    for at in range(4):  # the cache's tensors are on one device, or it is refused
        ts = [_OnDevice(x, 1 if i == at else 0) for i, x in enumerate((
            torch.zeros(4, 2, 16, 128, dtype=bf), torch.zeros(4, 2, 16, 128, dtype=bf), i32(2, 3), i32(2)))]
        with pytest.raises(ValueError, match="current CUDA device"):
            B.dsa_chunk_attn(B.paged_kv(*ts, 4), B.chunk(_OnDevice(i32(3), 0), _OnDevice(i32(2), 0), tokens=T),
                             _OnDevice(rows(4), 0), 0.1, _OnDevice(rows(4), 0), stream=stream)
    with pytest.raises(ValueError, match="one device"):
        B.chunk(_OnDevice(i32(3), 0), _OnDevice(i32(2), 1), tokens=4)


def test_rotary_takes_strided_axes(monkeypatch):
    """The axes of pairs may be a view: what the descriptor points to is their dense copy."""
    from dynamic_block_sparse_gb300 import binding as B
    monkeypatch.setattr(B, "_ptr", lambda t: None if t is None else t.data_ptr())
    axis = (torch.arange(128, dtype=torch.uint8) % 3)[::2]
    r = B.rotary(torch.arange(128, dtype=torch.int64)[::2], 128, axis,
                 torch.zeros(3, 5, dtype=torch.int32))
    assert (ctypes.c_uint8 * 64).from_address(r.axis)[:] == axis.tolist()
    assert (ctypes.c_int64 * 64).from_address(r.phase)[:] == list(range(0, 128, 2))


def test_a_cache_of_strided_or_other_tensors_is_refused(lib, monkeypatch):
    """The library reads the cache's tensors as dense arrays of its types: a slice of a wider page table
    would give each request another's pages."""
    import types

    from dynamic_block_sparse_gb300 import binding as B
    monkeypatch.setattr(B, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(B, "_on", lambda t, here: None if t is None else t.data_ptr())
    monkeypatch.setattr(B, "_current", lambda: -1)
    ran = []
    monkeypatch.setattr(B, "load", lambda: types.SimpleNamespace(**{n: lambda *a: ran.append(a) or 0 for n in (
        "dsa_append_chunk", "dsa_chunk_attn", "dsa_plan_chunk")}))
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t)
    bf, u8, stream = torch.bfloat16, torch.uint8, types.SimpleNamespace(cuda_stream=1)
    pool = lambda: z(4, 2, 16, 128, t=bf)
    good = dict(k_pages=pool(), v_pages=pool(), page_table=z(2, 3), seq_lens=z(2), num_q_heads=4,
                head_is_streaming=z(2, t=u8), status=z(1))
    chunk = B.chunk(z(3), z(2), z(6), z(6))

    def calls(kv):
        yield lambda: B.dsa_plan_chunk(kv, z(2), z(2), z(4), z(1), z(1), chunk, z(4), stream)
        yield lambda: B.dsa_append_chunk(kv, chunk, z(6, 2, 128, t=bf), z(6, 2, 128, t=bf), stream=stream)
        yield lambda: B.dsa_chunk_attn(kv, chunk, z(6, 4, 128, t=bf), 0.1, z(6, 4, 128, t=bf),
                                       workspace=z(4), stream=stream)

    for call in calls(B.paged_kv(**good)):
        call()
    assert len(ran) == 3
    for name, t in (("page_table", z(2, 6)[:, :3]), ("page_table", z(3, 2).t()), ("seq_lens", z(4)[::2]),
                    ("seq_lens", z(1)), ("k_pages", z(4, 4, 16, 128, t=bf)[:, ::2]),
                    ("v_pages", z(4, 2, 16, 256, t=bf)[..., ::2]),
                    ("v_pages", z(4, 2, 16, 128, t=torch.float16)), ("head_is_streaming", z(2)),
                    ("head_is_streaming", z(1, t=u8)), ("head_is_streaming", z(4, t=u8)[::2]),
                    ("status", z(1, t=torch.int64))):
        for call in calls(B.paged_kv(**{**good, name: t})):
            with pytest.raises(ValueError, match=name):
                call()
    kv, ws = B.paged_kv(**good), z(1).expand(1 << 20)  # (many bytes by its shape, four in memory)
    with pytest.raises(ValueError, match="workspace"):
        B.dsa_plan_chunk(kv, z(2), z(2), z(4), z(1), z(1), chunk, ws, stream)
    with pytest.raises(ValueError, match="workspace"):
        B.dsa_chunk_attn(kv, chunk, z(6, 4, 128, t=bf), 0.1, z(6, 4, 128, t=bf), workspace=ws,
                         stream=stream)
    assert len(ran) == 3


def test_plan_refuses_axes_beyond_its_indexes(lib):
    """The plan's indexes run a grid's step past the token axis and the stack: both stay below 2^31 by
    that."""
    def call(tokens, cap):
        return lib.dsa_plan_chunk(ctypes.byref(_kv()), 4096, 4096, 4096, cap, 4096, 4096,
                                  ctypes.byref(_chunk(tokens)), 8192, 0, None)
    most = (1 << 31) - 1 - (1 << 20)
    assert call(most + 1, 16) == -3 and call(16, most + 1) == -3 and call((1 << 31) - 1, 16) == -3
    assert call(most, most) == -5  # (these pass on to the workspace's check)


def test_plan_reference_takes_and_refuses():
    """The random steps above reach both outcomes."""
    seen = set()
    for seed in range(20):
        r = random.Random(seed)
        p, B, width, phys = 16, r.randint(1, 9), r.randint(2, 12), r.randint(6, 60)
        table = np.full((B, width), -7, dtype=np.int64)
        lens, free = [0] * B, list(range(phys))
        for _ in range(30):
            delta = [r.choice([0, 1, r.randint(1, p * 3), -r.randint(1, 40)]) for _ in range(B)]
            got = plan_reference(table, lens, delta, free, p, tokens=200)
            table, lens, free = got["table"], got["lens"], got["stack"]
            seen.add(got["refused"])
    assert seen == {True, False}
